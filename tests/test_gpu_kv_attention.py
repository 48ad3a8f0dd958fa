"""GPU: attention over the paged FP8 cache against the float64 oracle.

Bound, from the roundings on the way (A = sum_j p_j |v_j|, half steps of
fp16 2^-11, of bf16 2^-8, of fp32 2^-24; u = 2^-11 where one fp16 carries an
operand, 2^-21 where two do):
  scores   off by at most ds = smax * (uq + 2^-19) + 2^-22 (1 + |lse|), smax the
           largest scale * sum_c |q_c k_c|: the rounding of q to uq, products
           exact, at most 2 head_dim fp32 additions and three multiplications
  p        off by a factor e^(+-2 ds) and its rounding: 2 * 2 ds + up + 2^-20,
           with up = 2^-11 where out is bf16
  out      A * (the sum of those) + 2^-16 A for the fp32 sums over up to 2^12
           positions split over 64 lanes, and half a step of out's type;
           and, where fp16 holds p only to half its smallest step 2^-24 while the
           largest p is at least 2^7: 2^-25 / 2^7 = 2^-32 times sum_j |v_j|
  lse      2 ds + 2^-18
  weights  each p as above; the sum over n rows has n 2^-24 of itself
q is carried in 22 bits wherever it is not exact: uq = 2^-21."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x128_amd as fb
from gpu_helpers import dev, f32_of_store, host, say
from oracle import attention, formats
import workloads

pytestmark = pytest.mark.gpu

TENSOR, HEAD, CHANNEL = fb.KV_SCALE_TENSOR, fb.KV_SCALE_HEAD, fb.KV_SCALE_CHANNEL
SENTINEL = 77.25


class Problem:
    def __init__(self, seed, lens, news, H, Hk, D, bs, fmt=fb.E4M3, kind=HEAD, q_dt=fb.DT_BF16, spare=3, gap=0):
        rng = np.random.default_rng(seed)
        self.H, self.Hk, self.D, self.bs, self.fmt, self.kind, self.q_dt = H, Hk, D, bs, fmt, kind, q_dt
        self.lens, self.news = list(lens), list(news)
        B = len(lens)
        per = max(1, max(-(-n // bs) for n in lens)) + 1
        used = [-(-n // bs) for n in lens]
        blocks = sum(used) + spare
        order = rng.permutation(blocks)
        self.table = np.full((B, per), -1, np.int64)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.num_slots = blocks * bs
        # every code pattern in the pool, NaN and Inf among them, then finite codes where a sequence has positions
        finite = np.flatnonzero(np.isfinite(formats.decode(np.arange(256, dtype=np.uint8), fmt))).astype(np.uint8)
        small = finite[np.abs(formats.decode(finite, fmt)) <= (448 if fmt == fb.E4M3 else 64)]
        shape = (self.num_slots, Hk, D)
        self.k, self.v = rng.integers(0, 256, shape, dtype=np.uint8), rng.integers(0, 256, shape, dtype=np.uint8)
        for b, n in enumerate(lens):
            s = self.slots(b, n)
            self.k[s], self.v[s] = rng.choice(small, (n, Hk, D)), rng.choice(small, (n, Hk, D))
        n = {TENSOR: 1, HEAD: Hk, CHANNEL: Hk * D}[kind]
        self.ks = (rng.uniform(0.5, 2, n) / 64).astype(np.float32)
        self.vs = (rng.uniform(0.5, 2, n) / 64).astype(np.float32)
        self.starts = np.concatenate([[gap], gap + np.cumsum(news)]).astype(np.int64)
        self.tokens = int(self.starts[-1]) + gap
        q = rng.standard_normal((self.tokens, H, D)).astype(np.float32) * np.exp(rng.uniform(-2, 2, (self.tokens, H, 1))).astype(np.float32)
        self.q_store = workloads.f32_to_bf16_bits(q) if q_dt == fb.DT_BF16 else q
        self.scale = float(np.float32(D ** -0.5 / 4))

    def slots(self, b, n):
        j = np.arange(n)
        return self.table[b, j // self.bs] * self.bs + j % self.bs

    def device(self):
        return dict(q=dev(self.q_store), k_cache=dev(self.k), v_cache=dev(self.v), block_table=dev(self.table),
                    block_size=self.bs, q_starts=dev(self.starts), kv_lens=dev(np.array(self.lens, np.int64)),
                    k_scales=dev(self.ks), v_scales=dev(self.vs), fmt=self.fmt, scale_kind=self.kind,
                    max_q=max(max(self.news), 1), max_kv=max(max(self.lens), 1), softmax_scale=self.scale)

    def oracle(self, w_in=None):
        return attention.kv_attention(f32_of_store(self.q_store), self.k, self.v, self.table, self.bs, self.starts,
                                      self.lens, self.ks, self.vs, self.fmt, self.scale, w_in)


def _check(p, out, lse, want, w_out=None, w_in=None):
    out_bf16 = out.dtype == torch.bfloat16
    uq = 2.0 ** -21
    up = 2.0 ** -11 if out_bf16 else 2.0 ** -21
    o, l = f32_of_store(host(out)).astype(np.float64), host(lse).astype(np.float64)
    for b, w in enumerate(want):
        t0, t1 = w["tokens"]
        finite = np.isfinite(w["lse"])
        ds = w["smax"] * (uq + 2.0 ** -19) + 2.0 ** -22 * (1 + np.abs(np.where(finite, w["lse"], 0)))
        rel = 4 * ds + up + 2.0 ** -20 + 2.0 ** -16
        tol = w["absv"] * rel[..., None] + np.abs(w["out"]) * (2.0 ** -8 if out_bf16 else 2.0 ** -23) + 1e-30
        tol = tol + 2.0 ** -32 * np.repeat(w["sumv"], p.H // p.Hk, 0)
        err = np.abs(o[t0:t1] - w["out"])
        assert (err <= tol).all(), (b, "out", float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4].tolist())
        assert np.array_equal(np.isneginf(l[t0:t1]), ~finite), (b, "lse of rows that see nothing")
        le = np.abs(np.where(finite, l[t0:t1] - np.where(finite, w["lse"], 0), 0))
        assert (le <= 2 * ds + 2.0 ** -18).all(), (b, "lse", float(le.max()))
        if w_out is not None:
            n = p.lens[b]
            rows = (t1 - t0) * p.H // p.Hk
            base = np.zeros((p.Hk, n)) if w_in is None else w_in[b, :, :n].astype(np.float64)
            got, received = w_out[b, :, :n], w["weights"] - base
            r = 4 * (ds.max() if ds.size else 0) + 2.0 ** -18 + (rows + 1) * 2.0 ** -24
            wt = received * r + np.abs(w["weights"]) * 2.0 ** -23 + 1e-30
            we = np.abs(got - w["weights"])
            assert (we <= wt).all(), (b, "weights", float((we / wt).max()))


def _run(p, out_dtype=fb.DT_BF16, weights=False, w_in=True, **more):
    """One call into buffers filled with a sentinel, checked whole: what is not written stays."""
    d = p.device()
    d.update(more)
    out = torch.full((p.tokens, p.H, p.D), SENTINEL, dtype=torch.bfloat16 if out_dtype else torch.float32, device="cuda")
    lse = torch.full((p.tokens, p.H), SENTINEL, device="cuda")
    wi = wo = None
    if weights:
        wi = np.random.default_rng(5).uniform(0, 1, (len(p.lens), p.Hk, d["max_kv"] + 5)).astype(np.float32)
        wo = torch.full(wi.shape, SENTINEL, device="cuda")
        d.update(weights_in=dev(wi) if w_in else None, weights_out=wo)
        wi = wi if w_in else None
    got = fb.fp8_kv_attention(out=out, lse=lse, **d)
    assert got[0] is out and got[1] is lse
    torch.cuda.synchronize()
    w_host = None if wo is None else host(wo).astype(np.float64)
    _check(p, out, lse, p.oracle(wi), w_host, wi)
    a, b = int(p.starts[0]), int(p.starts[-1])
    for x in (out, lse):
        assert (x[:a] == SENTINEL).all() and (x[b:] == SENTINEL).all(), "rows of no sequence were written"
    if wo is not None:
        for i, n in enumerate(p.lens):
            assert (w_host[i, :, n:] == SENTINEL).all(), "weights behind the last position were written"
    return out, lse, wo


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,kind,q_dt", [(0, HEAD, 1), (0, CHANNEL, 1), (1, TENSOR, 1), (1, CHANNEL, 0), (0, TENSOR, 0)])
def test_decode_step(D, fmt, kind, q_dt):
    say(f"decode D={D} fmt={fmt} kind={kind} q_dt={q_dt}")
    p = Problem(11 + D + fmt, [1, 2, 31, 32, 33, 64, 100, 257], [1] * 8, 8, 2, D, 16, fmt, kind, q_dt)
    _run(p)
    _run(p, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,kind,q_dt", [(0, HEAD, 1), (0, CHANNEL, 1), (1, TENSOR, 1), (1, CHANNEL, 0), (0, TENSOR, 0)])
def test_chunk(D, fmt, kind, q_dt):
    say(f"chunk D={D} fmt={fmt} kind={kind} q_dt={q_dt}")
    p = Problem(21 + D + fmt, [70, 200, 1, 333, 65], [70, 37, 1, 129, 64], 4, 2, D, 16, fmt, kind, q_dt)
    _run(p)
    _run(p, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("H,Hk", [(1, 1), (7, 1), (12, 4), (16, 1), (34, 2), (40, 1)])
@pytest.mark.parametrize("new", [1, 3, 9])
def test_shared_heads(H, Hk, new):
    """Group sizes on both sides of every tile, powers of two and not."""
    say(f"shared heads {H}/{Hk} new={new}")
    _run(Problem(H + 100 * new, [50, 130, new], [new, max(1, new - 1), new], H, Hk, 64, 8, kind=CHANNEL), weights=True)


@pytest.mark.parametrize("bs", [1, 3, 7, 16, 48, 128, 1000])
@pytest.mark.parametrize("new", [1, 40])
def test_block_sizes(bs, new):
    """Pages that end inside a tile, slot lists, and pages longer than a sequence."""
    say(f"block size {bs} new={new}")
    _run(Problem(bs, [new, 95, 200], [new, new, 1], 4, 2, 64, bs, kind=HEAD))


@pytest.mark.parametrize("new,D,kind,q_dt", [(1, 128, HEAD, 1), (1, 64, CHANNEL, 0), (5, 64, CHANNEL, 1), (5, 256, HEAD, 1),
                                             (90, 128, CHANNEL, 1), (90, 64, TENSOR, 0), (90, 256, CHANNEL, 1)])
@pytest.mark.parametrize("w_in", [False, True])
def test_weights(new, D, kind, q_dt, w_in):
    say(f"weights new={new} D={D} kind={kind} w_in={w_in}")
    _run(Problem(31 + new, [new, 97, 300, 640], [new, max(1, new - 3), 1, new], 6, 2, D, 16, kind=kind, q_dt=q_dt),
         weights=True, w_in=w_in)


def test_weights_accumulate_in_place():
    p = Problem(41, [60, 130], [2, 2], 4, 2, 64, 16)
    d = p.device()
    w = torch.zeros((2, 2, 130), device="cuda")
    for _ in range(3):
        fb.fp8_kv_attention(weights_in=w, weights_out=w, **d)
    once = torch.zeros_like(w)
    fb.fp8_kv_attention(weights_out=once, **d)
    torch.cuda.synchronize()
    assert torch.equal(w[1], (once[1] + once[1]) + once[1])
    # every query row gives one unit of weight
    assert torch.allclose(once.sum(-1).cpu(), torch.full((2, 2), 4.0), atol=1e-4)


@pytest.mark.parametrize("max_q", [0, 1, 60])
def test_weights_of_a_call_without_queries(max_q):
    """No query token anywhere: the weights come through, and rows behind a sequence's end stay."""
    p = Problem(45, [60, 0, 130], [0, 0, 0], 4, 2, 64, 16)
    wi = torch.rand((3, 2, 140), device="cuda")
    wo = torch.full((3, 2, 140), SENTINEL, device="cuda")
    d = p.device()
    d.update(max_q=max_q)
    fb.fp8_kv_attention(weights_in=wi, weights_out=wo, **d)
    torch.cuda.synchronize()
    for b, n in enumerate(p.lens):
        assert torch.equal(wo[b, :, :n], wi[b, :, :n]) and (wo[b, :, n:] == SENTINEL).all()


@pytest.mark.parametrize("new", [1, 2, 50])
def test_rows_that_see_nothing(new):
    """Sequences of no positions, fewer positions than new tokens, all pages dropped, and no new tokens."""
    say(f"empty rows new={new}")
    p = Problem(51, [0, new // 2, 80, 100, 33], [new, new, new, 0, new], 4, 2, 128, 16)
    p.table[2, :] = -1
    _run(p, weights=True)
    _run(p, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("new", [1, 40])
def test_dropped_and_bad_pages(new):
    """Entries of -1, past the pool, and far out of range are left out, the last page's end past the pool too."""
    say(f"dropped pages new={new}")
    p = Problem(61, [200, 150, 90], [new, new, new], 4, 2, 128, 16)
    p.table[0, [0, 3, 7]] = [-1, p.num_slots // 16, 1 << 40]
    p.table[1, 4] = -(1 << 62)
    p.table[2, 1] = (1 << 63) - 1
    _run(p, weights=True)
    q = Problem(62, [48, 48], [new, new], 4, 2, 64, 16, spare=0)
    last = int(np.argwhere(q.table[0] == q.table.max())[0][0]) if (q.table[0] == q.table.max()).any() else -1
    cut = 5
    q.num_slots -= cut                       # the pool ends inside its last page
    q.k, q.v = q.k[:q.num_slots].copy(), q.v[:q.num_slots].copy()
    assert last >= -1
    _run(q)


@pytest.mark.parametrize("new", [1, 64])
def test_shared_pages(new):
    """Two sequences on the same pages, and one page twice in a sequence: each has its own result and weights."""
    p = Problem(71, [128, 128, 128], [new, new, new], 4, 2, 64, 16)
    p.table[1, :4] = p.table[0, :4]
    p.table[2, 1] = p.table[2, 0]
    _run(p, weights=True)


@pytest.mark.parametrize("new", [1, 33])
def test_strided_queries(new):
    """q as the query slice of a fused projection output, and tokens in front of and behind the sequences."""
    p = Problem(81, [new, 77], [new, new], 8, 2, 128, 16, gap=2)
    rng = np.random.default_rng(1)
    fused = workloads.f32_to_bf16_bits(rng.standard_normal((p.tokens, 12 * 128)).astype(np.float32))
    p.q_store = fused[:, :8 * 128].reshape(p.tokens, 8, 128)
    _run(p, q=dev(fused)[:, :8 * 128].view(p.tokens, 8, 128))


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("weights", [False, True])
def test_long_split_cache(new, weights):
    """One long sequence beside short ones, split over its positions."""
    say(f"long cache new={new} weights={weights}")
    _run(Problem(91, [9001, 5, 1300], [new, min(new, 5), new], 4, 1, 64, 16, kind=CHANNEL), weights=weights)


@pytest.mark.parametrize("new", [1, 40])
def test_lengths_below_the_bounds(new):
    """max_q and max_kv are upper bounds: a larger one changes the split, not the result."""
    p = Problem(101, [300, 40], [new, new], 4, 2, 128, 16)
    more = 128 * 16
    p.table = np.concatenate([p.table, np.full((2, 128), -1, np.int64)], 1)
    _run(p, max_q=new + 3, max_kv=more)
    _run(p, max_q=2 * new + 40, max_kv=300, weights=True)


@pytest.mark.parametrize("new", [3, 30])
def test_tokens_past_max_q_are_left(new):
    p = Problem(103, [300, 40], [new, new], 8, 2, 64, 16, kind=CHANNEL)
    d = p.device()
    ref, ref_lse = fb.fp8_kv_attention(**d)
    d["max_q"] = new - 2
    out, lse = torch.full_like(ref, SENTINEL), torch.full_like(ref_lse, SENTINEL)
    fb.fp8_kv_attention(out=out, lse=lse, **d)
    torch.cuda.synchronize()
    tol = 2.0 ** -7 * ref.float().abs().max()
    for b in (0, 1):
        a = b * new
        assert (out[a:a + new - 2].float() - ref[a:a + new - 2].float()).abs().max() <= tol
        assert (out[a + new - 2:a + new] == SENTINEL).all() and (lse[a + new - 2:a + new] == SENTINEL).all()


@pytest.mark.parametrize("new", [1, 40])
def test_pool_without_slots(new):
    p = Problem(104, [70, 50], [new, new], 4, 2, 64, 16)
    p.table[:] = 0
    p.num_slots, p.k, p.v = 0, p.k[:0], p.v[:0]
    out, lse, _ = _run(p, weights=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("new", [1, 5, 40])
def test_slots_past_four_gigabytes(new):
    """Row offsets of 32 bits would wrap: pages at both ends of a pool of 4.3 GB a cache."""
    p = Problem(106, [100, 180], [new, new], 16, 8, 128, 16, kind=HEAD)
    d = p.device()
    ref, ref_lse = fb.fp8_kv_attention(**d)
    slots = (1 << 32) // 1024 + 4096
    big = {}
    for name in ("k_cache", "v_cache"):
        big[name] = torch.zeros((slots, 8, 128), dtype=torch.uint8, device="cuda")
        big[name][-p.num_slots:] = d[name]
    table = torch.where(d["block_table"] >= 0, d["block_table"] + (slots - p.num_slots) // 16, d["block_table"])
    out, lse = fb.fp8_kv_attention(**{**d, **big, "block_table": table})
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, over the same cache."""
    p = Problem(108, [5000, 900], [1, 1], 8, 2, 128, 16, kind=CHANNEL)
    q = Problem(108, [5000, 900], [60, 40], 8, 2, 128, 16, kind=CHANNEL)
    dp, dq = p.device(), q.device()
    ref_p, ref_q = fb.fp8_kv_attention(**dp)[0], fb.fp8_kv_attention(**dq)[0]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((fb.fp8_kv_attention(stream=a, **dp)[0], fb.fp8_kv_attention(stream=b, **dq)[0]))
    default = fb.fp8_kv_attention(stream=0, **dp)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref_p) and torch.equal(y, ref_q) for x, y in got) and torch.equal(default, ref_p)


@pytest.mark.parametrize("Hk,batch,max_kv", [(8, 2, 16384), (4, 4, 20000), (2, 4, 32768), (6, 2, 65536), (8, 1, 131072)])
@pytest.mark.parametrize("D,new", [(64, 1), (128, 3), (256, 1)])
def test_many_workgroups(Hk, batch, max_kv, D, new):
    """Bounds so large that a workgroup takes two or four neighbouring heads, over short and empty sequences."""
    say(f"many workgroups Hk={Hk} batch={batch} max_kv={max_kv} D={D} new={new}")
    lens = [700, 33, 0, 260][:batch]
    p = Problem(107 + Hk, lens, [new] * batch, 4 * Hk, Hk, D, 64, kind=CHANNEL)
    p.table = np.concatenate([p.table, np.full((batch, -(-max_kv // 64)), -1, np.int64)], 1)
    _run(p, max_kv=max_kv, weights=True)
    _run(p, max_kv=max_kv, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("fmt", [fb.E4M3, fb.E5M2])
@pytest.mark.parametrize("new,D", [(2, 64), (3, 128), (7, 128), (4, 256), (40, 64), (70, 128), (150, 256)])
def test_values_that_are_not_finite(new, D, fmt):
    """NaN (and Inf) codes among the new tokens' keys or values: rows in front of them are as without, rows that
    see a value's get exactly its NaN or Inf in that channel."""
    say(f"not finite new={new} D={D} fmt={fmt}")
    lens = [new + 90, new]
    clean = Problem(113 + new, lens, [new, new], 8, 2, D, 16, fmt, HEAD)
    ref, _ = fb.fp8_kv_attention(**clean.device())
    bad = Problem(113 + new, lens, [new, new], 8, 2, D, 16, fmt, HEAD)
    at = new // 2 + 1 if new > 2 else 1                     # the new token whose states are not finite
    for b in (0, 1):
        s = bad.slots(b, lens[b])[lens[b] - new + at]
        bad.v[s, 0, 5] = 0x7F
        bad.v[s, 1, D - 1] = 0xFF if fmt == fb.E4M3 else 0xFC   # NaN, or -Inf
    out, _ = fb.fp8_kv_attention(**bad.device())
    torch.cuda.synchronize()
    for b in (0, 1):
        t0 = b * new
        assert torch.equal(out[t0:t0 + at], ref[t0:t0 + at]), "rows that do not see the value"
        seen, was = out[t0 + at:t0 + new].float(), ref[t0 + at:t0 + new].float()
        assert torch.isnan(seen[:, :4, 5]).all()
        assert (torch.isnan(seen[:, 4:, D - 1]).all() if fmt == fb.E4M3 else (seen[:, 4:, D - 1] == -torch.inf).all())
        keep = torch.ones(8, D, dtype=torch.bool)
        keep[:4, 5] = keep[4:, D - 1] = False
        assert torch.equal(seen[:, keep], was[:, keep]), "channels that are finite"
    # keys: a row that sees a NaN key is NaN throughout, one that does not is as without
    bad = Problem(113 + new, lens, [new, new], 8, 2, D, 16, fmt, HEAD)
    bad.k[bad.slots(0, lens[0])[lens[0] - new + at], :, 3] = 0x7F
    out, lse = fb.fp8_kv_attention(**bad.device())
    torch.cuda.synchronize()
    assert torch.equal(out[:at], ref[:at]) and torch.equal(out[new:], ref[new:])
    assert torch.isnan(out[at:new].float()).all() and torch.isnan(lse[at:new]).all()


def test_extreme_queries():
    """Rows of zeros, of the largest and of subnormal values: each row has its own power of two."""
    p = Problem(111, [65] * 4, [1] * 4, 4, 2, 128, 16, kind=CHANNEL)
    q = f32_of_store(p.q_store).copy()
    q[0] = 0
    q[1] *= 2.0 ** 60
    q[2] *= 2.0 ** -100
    q[3, 0, 1:] *= 2.0 ** -30
    p.q_store = workloads.f32_to_bf16_bits(q)
    p.ks = (p.ks * np.float32(2.0 ** -64)).astype(np.float32)
    _run(p)
    p.q_dt, p.q_store = fb.DT_F32, q
    _run(p, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kind,power", [(HEAD, -64), (TENSOR, -120), (CHANNEL, -64)])
def test_vanishing_scores(new, kind, power):
    """Tiny queries under tiny scales: the factor of a row underflows, the masked positions stay masked."""
    p = Problem(117, [new + 30, new], [new, new], 4, 2, 64, 16, kind=kind)
    q = f32_of_store(p.q_store) * np.float32(2.0 ** -120)
    p.q_store = workloads.f32_to_bf16_bits(q)
    p.ks = np.maximum(p.ks * np.float32(2.0 ** power), np.float32(2.0 ** -126))
    _run(p, weights=True)
    _run(p, out_dtype=fb.DT_F32)


@pytest.mark.parametrize("new", [1, 5, 40, 150])
@pytest.mark.parametrize("weights", [False, True])
def test_without_lse(new, weights):
    """The C call with no lse pointer gives the same outputs and weights."""
    p = Problem(119, [3000, new], [new, new], 8, 2, 64, 16, kind=CHANNEL)
    d = p.device()
    w = [torch.zeros((2, 2, 3000), device="cuda") for _ in range(2)] if weights else [None, None]
    ref, _ = fb.fp8_kv_attention(weights_out=w[0], **d)
    lib, out = fb.load_library(), torch.empty_like(ref)
    need = lib.fp8_kv_attention_workspace_bytes(p.tokens, 8, 2, 64, 2, new, 3000, weights)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    st = lib.fp8_kv_attention(d["q"].data_ptr(), 1, p.tokens, 8, 2, 64, 512, d["k_cache"].data_ptr(), d["v_cache"].data_ptr(),
                              p.num_slots, d["block_table"].data_ptr(), p.table.shape[1], 16, 2, d["q_starts"].data_ptr(),
                              d["kv_lens"].data_ptr(), new, 3000, p.fmt, p.kind, d["k_scales"].data_ptr(),
                              d["v_scales"].data_ptr(), p.scale, out.data_ptr(), 1, None, None,
                              w[1].data_ptr() if weights else None, 3000 if weights else 0, ws.data_ptr(), ws.numel(),
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(out, ref)
    assert not weights or torch.equal(w[0], w[1])


def test_large_scores_do_not_overflow():
    """Scores in the thousands, rising and falling along the cache: the running maximum has to follow."""
    for new in (1, 40):
        p = Problem(121, [900], [new], 4, 2, 64, 16)
        s = p.slots(0, 900)
        p.k[s] = 0x38                                               # 1.0
        ramp = formats.encode_nearest(np.concatenate([np.linspace(0, 400, 450), np.linspace(400, -400, 450)]), 0)
        p.k[s, :, 0] = np.asarray(ramp, np.uint8)[:, None]
        q = np.zeros((p.tokens, 4, 64), np.float32)
        q[:, :, 0] = 64.0
        q[:, :, 1] = 1.0
        p.q_store, p.ks = workloads.f32_to_bf16_bits(q), np.ones(2, np.float32)
        _run(p, weights=True)


def test_equal_calls_give_equal_bits_on_another_stream_and_captured():
    for new, lens in ((1, [700, 90]), (45, [300, 45])):
        p = Problem(131, lens, [new, new], 8, 2, 128, 16, kind=CHANNEL)
        d = p.device()
        w0 = torch.zeros((2, 2, max(lens)), device="cuda")
        ref, ref_lse = fb.fp8_kv_attention(weights_out=w0, **d)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        w1 = torch.zeros_like(w0)
        out, lse = fb.fp8_kv_attention(weights_out=w1, stream=side, **d)
        side.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse) and torch.equal(w1, w0)
        out, lse = fb.fp8_kv_attention(stream=side.cuda_stream, **d)
        side.synchronize()
        assert torch.equal(lse, ref_lse) or p.kind == CHANNEL
        # captured: the lengths are read on the device at each replay
        bytes_ = fb.fp8_kv_attention_workspace_bytes(p.tokens, 8, 2, 128, 2, new, max(lens), True)
        ws = torch.empty(max(bytes_, 16), dtype=torch.uint8, device="cuda")
        out2, lse2, w2 = torch.empty_like(ref), torch.empty_like(ref_lse), torch.zeros_like(w0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fb.fp8_kv_attention(out=out2, lse=lse2, weights_out=w2, workspace=ws, **d)
        for _ in range(3):
            out2.fill_(SENTINEL)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out2, ref) and torch.equal(lse2, ref_lse) and torch.equal(w2, w0)
        d["kv_lens"].copy_(torch.tensor([lens[0] - 40, lens[1]], device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        ref3, _ = fb.fp8_kv_attention(weights_out=torch.zeros_like(w0), **d)
        torch.cuda.synchronize()
        assert torch.equal(out2, ref3) and not torch.equal(out2, ref)


def test_binding_refuses_what_the_library_cannot_see():
    p = Problem(141, [40], [1], 4, 2, 64, 16)
    d = p.device()
    for key, bad in (("kv_lens", d["kv_lens"].int()), ("block_table", d["block_table"].int()), ("k_cache", d["k_cache"].view(torch.int8))):
        with pytest.raises(TypeError):
            fb.fp8_kv_attention(**{**d, key: bad})
    for key, bad in (("v_cache", d["v_cache"][:-1]), ("q_starts", d["q_starts"][:-1]), ("kv_lens", d["kv_lens"].cpu()),
                     ("k_scales", d["k_scales"][:1]), ("block_table", torch.zeros((1, 8), dtype=torch.int64, device="cuda")[:, ::2]),
                     ("q", d["q"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            fb.fp8_kv_attention(**{**d, key: bad})
    with pytest.raises(ValueError):
        fb.fp8_kv_attention(weights_in=torch.zeros(1, 2, 40, device="cuda"), **d)
    with pytest.raises(ValueError):
        fb.fp8_kv_attention(weights_out=torch.zeros(1, 4, 40, device="cuda"), **d)
    with pytest.raises(fb.Fp8Error):
        fb.fp8_kv_attention(weights_out=torch.zeros(1, 2, 39, device="cuda"), **d)
    with pytest.raises(fb.Fp8Error):
        fb.fp8_kv_attention(**{**d, "max_kv": 64 + 16})
