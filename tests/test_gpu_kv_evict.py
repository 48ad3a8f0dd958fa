"""GPU: the choice of positions to keep and their move, against the oracle,
exactly: positions, counts, every byte of both pools and every weight."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x128_amd as fb
import workloads
from gpu_helpers import assert_codes_equal, dev, host, say
from oracle import attention, quant

pytestmark = pytest.mark.gpu


def _weights(rng, shape, kind):
    if kind == "heavy":
        return np.exp(2 * rng.standard_normal(shape) - 4).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 3, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    w = rng.standard_normal(shape).astype(np.float32)              # signs, zeros of both signs, Inf and NaN
    w[rng.random(shape) < 0.2] = 0.0
    w[rng.random(shape) < 0.1] = -0.0
    w[rng.random(shape) < 0.02] = np.inf
    w[rng.random(shape) < 0.02] = -np.inf
    w[rng.random(shape) < 0.02] = np.nan
    return w


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "odd"])
@pytest.mark.parametrize("kv_heads,top,keep,first,recent", [
    (1, 1, 1, 0, 0), (1, 5, 2, 1, 1), (2, 64, 63, 0, 0), (8, 1000, 300, 4, 64), (3, 1025, 1024, 0, 1024),
    (4, 2500, 1, 0, 0), (2, 2500, 7, 7, 0), (1, 20001, 9000, 4, 100), (2, 300, 0, 0, 0), (2, 300, 400, 100, 300)])
def test_select(kind, kv_heads, top, keep, first, recent):
    say(f"select {kind} kv_heads={kv_heads} top={top} keep={keep} first={first} recent={recent}")
    rng = np.random.default_rng(top + keep)
    lens = np.array([top, 0, min(top, keep), min(top, keep + 1), max(1, top // 2), rng.integers(0, top + 1)], np.int64)
    w = _weights(rng, (lens.size, kv_heads, top + 3), kind)
    kept = torch.full((lens.size, keep), -77, dtype=torch.int64, device="cuda")
    got, got_lens = fb.fp8_kv_evict_select(dev(w), dev(lens), keep, first=first, recent=recent, max_kv=top, kept=kept)
    torch.cuda.synchronize()
    want, want_lens = attention.evict_select(w, lens, keep, first, recent)
    assert np.array_equal(host(got_lens), want_lens)
    assert np.array_equal(host(got), want), np.argwhere(host(got) != want)[:5]


def test_select_lengths_are_clamped():
    w = _weights(np.random.default_rng(1), (3, 2, 50), "heavy")
    lens = np.array([60, -5, 1 << 40], np.int64)
    got, n = fb.fp8_kv_evict_select(dev(w), dev(lens), 10)
    want, want_n = attention.evict_select(w, [50, 0, 50], 10, 0, 0)
    torch.cuda.synchronize()
    assert np.array_equal(host(got), want) and np.array_equal(host(n), want_n)


def _cache(rng, slots, heads, D):
    return rng.integers(0, 256, (slots, heads, D), dtype=np.uint8)


def _table(rng, batch, per, blocks):
    return rng.permutation(blocks)[:batch * per].reshape(batch, per).astype(np.int64)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("heads,D,bs", [(2, 64, 16), (8, 128, 16), (1, 16, 1), (3, 80, 5), (2, 576, 64), (1, 256, 1000)])
@pytest.mark.parametrize("top,keep", [(1, 1), (70, 30), (700, 699), (3000, 1400)])
def test_compact(in_place, heads, D, bs, top, keep):
    say(f"compact in_place={in_place} heads={heads} D={D} bs={bs} top={top} keep={keep}")
    rng = np.random.default_rng(top + D)
    lens = np.array([top, 0, min(top, keep), max(1, top - 1)], np.int64)
    B, per, per_to = lens.size, -(-top // bs), -(-keep // bs)
    blocks = B * (per + per_to) + 2
    table = _table(rng, B, per + per_to, blocks)
    src = np.ascontiguousarray(table[:, :per])
    dst = src if in_place else np.ascontiguousarray(table[:, per:])
    w = _weights(rng, (B, heads, top), "heavy")
    kept, kept_lens = attention.evict_select(w, lens, keep, 0, 0)
    k, v = _cache(rng, blocks * bs, heads, D), _cache(rng, blocks * bs, heads, D)
    kd, vd, sd = dev(k), dev(v), dev(src)
    wi = dev(w)
    wo = wi if in_place else torch.full((B, heads, keep), -7.0, device="cuda")
    fb.fp8_kv_compact(kd, vd, sd, sd if in_place else dev(dst), bs, dev(kept), dev(kept_lens), weights_in=wi,
                      weights_out=wo)
    torch.cuda.synchronize()
    assert_codes_equal(host(kd), attention.compact(k, src, dst, bs, kept, kept_lens), "k")
    assert_codes_equal(host(vd), attention.compact(v, src, dst, bs, kept, kept_lens), "v")
    want = w.copy() if in_place else np.full((B, heads, keep), -7.0, np.float32)
    for b in range(B):
        n = int(kept_lens[b])
        want[b, :, :n] = w[b][:, kept[b, :n]]
    assert np.array_equal(host(wo), want)


@pytest.mark.parametrize("heads,D,bs", [(2, 64, 16), (8, 128, 16), (1, 16, 1), (3, 80, 5), (2, 576, 64)])
@pytest.mark.parametrize("top,keep", [(70, 30), (700, 699), (3000, 1400)])
def test_compact_in_place_by_the_tables_values(heads, D, bs, top, keep):
    """The same pages in the same places, named by another, shorter table: all of them, only the first or the last,
    or none, a different choice each sequence."""
    say(f"compact by values heads={heads} D={D} bs={bs} top={top} keep={keep}")
    rng = np.random.default_rng(top + D + 1)
    lens = np.array([top, top - 1, top, max(keep + 1, top - 7)], np.int64)
    B, per, per_to = lens.size, -(-top // bs), -(-keep // bs)
    blocks = B * (per + per_to) + 2
    table = _table(rng, B, per + per_to, blocks)
    src, dst = np.ascontiguousarray(table[:, :per]), np.ascontiguousarray(table[:, per:])
    dst[0] = src[0, :per_to]
    dst[1, 0] = src[1, 0]
    dst[2, per_to - 1] = src[2, per_to - 1]
    w = _weights(rng, (B, heads, top), "heavy")
    kept, kept_lens = attention.evict_select(w, lens, keep, 0, 0)
    k, v = _cache(rng, blocks * bs, heads, D), _cache(rng, blocks * bs, heads, D)
    kd, vd, wo = dev(k), dev(v), torch.full((B, heads, keep), -7.0, device="cuda")
    fb.fp8_kv_compact(kd, vd, dev(src), dev(dst), bs, dev(kept), dev(kept_lens), weights_in=dev(w), weights_out=wo)
    torch.cuda.synchronize()
    assert_codes_equal(host(kd), attention.compact(k, src, dst, bs, kept, kept_lens), "k")
    assert_codes_equal(host(vd), attention.compact(v, src, dst, bs, kept, kept_lens), "v")
    want = np.full((B, heads, keep), -7.0, np.float32)
    for b in range(B):
        n = int(kept_lens[b])
        want[b, :, :n] = w[b][:, kept[b, :n]]
    assert np.array_equal(host(wo), want)


def test_compact_bad_entries_leave_the_destination():
    """Positions and pages outside their table or pool, on either side; counts past the row; short destinations."""
    rng = np.random.default_rng(9)
    bs, heads, D = 4, 2, 32
    src = np.array([[3, -1, 1 << 40, 0], [2, 4, 9, -(1 << 50)]], np.int64)
    dst = np.array([[5, 6], [-1, 7]], np.int64)
    kept = np.array([[0, 2, 5, 9, 13, 15, 16, 1 << 33, -1, 14], [1, 3, 4, 6, 8, 11, 12, 15, 2, 3]], np.int64)
    kept_lens = np.array([99, 8], np.int64)
    k, v = _cache(rng, 31, heads, D), _cache(rng, 31, heads, D)         # block 7 ends past the pool
    w = rng.random((2, heads, 10)).astype(np.float32)
    kd, vd, wo = dev(k), dev(v), torch.full((2, heads, 9), -7.0, device="cuda")
    fb.fp8_kv_compact(kd, vd, dev(src), dev(dst), bs, dev(kept), dev(kept_lens), weights_in=dev(w), weights_out=wo)
    torch.cuda.synchronize()
    assert_codes_equal(host(kd), attention.compact(k, src, dst, bs, kept, kept_lens), "k")
    assert_codes_equal(host(vd), attention.compact(v, src, dst, bs, kept, kept_lens), "v")
    want = np.full((2, heads, 9), -7.0, np.float32)
    for b, n in ((0, 9), (1, 8)):
        for i in range(n):
            if 0 <= kept[b, i] < 10:
                want[b, :, i] = w[b, :, kept[b, i]]
    assert np.array_equal(host(wo), want)


def test_from_prompt_to_eviction_and_on():
    """The operators as a server uses them: a prompt's attention, its states
    appended, decode steps that collect the weights, an eviction in place, and
    further steps over what was kept."""
    rng = np.random.default_rng(17)
    H, Hk, D, bs, lens, keep = 8, 2, 64, 16, [150, 90], 64
    B, per = 2, 12
    table_np = _table(rng, B, per, 30)
    table = dev(table_np)
    scales = torch.full((Hk,), 4 / 448, device="cuda")
    kc, vc = (torch.zeros((30 * bs, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    starts = np.array([0, 150, 240], np.int64)
    qkv = torch.from_numpy(rng.standard_normal((240, (H + 2 * Hk) * D)).astype(np.float32)).cuda().to(torch.bfloat16)
    q, k, v = qkv[:, :H * D].view(240, H, D), qkv[:, H * D:(H + Hk) * D].view(240, Hk, D), qkv[:, (H + Hk) * D:].view(240, Hk, D)
    out, lse = fb.fp8_prompt_attention(q, k, v, dev(starts), max_len=150)

    def slots(b, j):
        return table_np[b, j // bs] * bs + j % bs

    at = dev(np.concatenate([slots(b, np.arange(n)) for b, n in enumerate(lens)]))
    fb.fp8_kv_append(k, at, kc, scales, fb.E4M3, fb.KV_SCALE_HEAD)
    fb.fp8_kv_append(v, at, vc, scales, fb.E4M3, fb.KV_SCALE_HEAD)
    w = torch.zeros((B, Hk, per * bs), device="cuda")
    n = np.array(lens, np.int64)
    # the same prompt through the cache: within what E4M3 states are off by (2^-4 each of k and v)
    chunk, _ = fb.fp8_kv_attention(q, kc, vc, table, bs, dev(starts), dev(n), scales, scales, fb.E4M3, fb.KV_SCALE_HEAD,
                                   max_q=150, max_kv=per * bs, weights_in=w, weights_out=w)
    torch.cuda.synchronize()
    rel = (chunk.float() - out.float()).norm() / out.float().norm()
    assert rel < 0.1, float(rel)
    assert torch.allclose(w.sum((1, 2)).cpu(), torch.tensor([150.0 * H, 90.0 * H]), rtol=1e-4)

    def step(kc_np, vc_np, n, w_np):
        """A decode step on the GPU and in the oracle, weights in place."""
        new = torch.from_numpy(rng.standard_normal((B, (H + 2 * Hk) * D)).astype(np.float32)).cuda().to(torch.bfloat16)
        qn, kn, vn = new[:, :H * D].view(B, H, D), new[:, H * D:(H + Hk) * D].view(B, Hk, D), new[:, (H + Hk) * D:].view(B, Hk, D)
        s = np.array([slots(b, int(n[b])) for b in range(B)])
        fb.fp8_kv_append(kn, dev(s), kc, scales, fb.E4M3, fb.KV_SCALE_HEAD)
        fb.fp8_kv_append(vn, dev(s), vc, scales, fb.E4M3, fb.KV_SCALE_HEAD)
        sc = host(scales)
        for pool, x in ((kc_np, kn), (vc_np, vn)):
            x32 = x.float().cpu().numpy()
            pool[:] = quant.kv_append(pool, x32, s, fb.KV_SCALE_HEAD, sc, fb.E4M3)
        n = n + 1
        w_d = w
        for b in range(B):
            w_d[b, :, int(n[b]) - 1] = 0
            w_np[b, :, int(n[b]) - 1] = 0
        got, _ = fb.fp8_kv_attention(qn, kc, vc, table, bs, dev(np.arange(B + 1, dtype=np.int64)), dev(n), scales, scales,
                                     fb.E4M3, fb.KV_SCALE_HEAD, max_q=1, max_kv=per * bs, weights_in=w_d, weights_out=w_d)
        torch.cuda.synchronize()
        want = attention.kv_attention(qn.float().cpu().numpy(), kc_np, vc_np, table_np, bs, np.arange(B + 1), n, sc, sc,
                                      fb.E4M3, D ** -0.5, w_np)
        for b in range(B):
            tol = want[b]["absv"][0] * 2.0 ** -9 + np.abs(want[b]["out"][0]) * 2.0 ** -8
            assert (np.abs(got[b].float().cpu().numpy() - want[b]["out"][0]) <= tol).all()
            w_np[b, :, :int(n[b])] = want[b]["weights"]
        assert np.allclose(host(w), w_np, rtol=1e-4, atol=1e-5)
        return n

    kc_np, vc_np, w_np = host(kc).copy(), host(vc).copy(), host(w).astype(np.float64)
    for _ in range(2):
        n = step(kc_np, vc_np, n, w_np)
    before = host(w).copy()
    kept, kept_lens = fb.fp8_kv_evict_select(w, dev(n), keep, first=2, recent=8, max_kv=per * bs)
    fb.fp8_kv_compact(kc, vc, table, table, bs, kept, kept_lens, weights_in=w, weights_out=w)
    torch.cuda.synchronize()
    want_kept, want_lens = attention.evict_select(before, n, keep, 2, 8)
    assert np.array_equal(host(kept), want_kept) and np.array_equal(host(kept_lens), want_lens)
    kc_np[:] = attention.compact(kc_np, table_np, table_np, bs, want_kept, want_lens)
    vc_np[:] = attention.compact(vc_np, table_np, table_np, bs, want_kept, want_lens)
    assert_codes_equal(host(kc), kc_np, "k after eviction")
    assert_codes_equal(host(vc), vc_np, "v after eviction")
    w_np[:] = host(w)
    n = want_lens.copy()
    for _ in range(3):
        n = step(kc_np, vc_np, n, w_np)


def test_captured_and_replayed():
    rng = np.random.default_rng(23)
    bs, heads, D, top, keep, B = 16, 2, 64, 500, 200, 3
    per, per_to = -(-top // bs), -(-keep // bs)
    table = _table(rng, B, per + per_to, B * (per + per_to))
    src, dst = np.ascontiguousarray(table[:, :per]), np.ascontiguousarray(table[:, per:])
    w, lens = _weights(rng, (B, heads, top), "heavy"), np.array([500, 123, 300], np.int64)
    k, v = _cache(rng, table.size * bs, heads, D), _cache(rng, table.size * bs, heads, D)
    kd, vd, wd, ld, sd, dd = dev(k), dev(v), dev(w), dev(lens), dev(src), dev(dst)
    kept, kl = torch.zeros((B, keep), dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    ws = torch.empty(fb.fp8_kv_evict_select_workspace_bytes(B, top), dtype=torch.uint8, device="cuda")
    wo = torch.zeros((B, heads, keep), device="cuda")

    def call():
        fb.fp8_kv_evict_select(wd, ld, keep, first=4, recent=20, kept=kept, kept_lens=kl, workspace=ws)
        fb.fp8_kv_compact(kd, vd, sd, dd, bs, kept, kl, weights_in=wd, weights_out=wo)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in range(3):
        w = _weights(np.random.default_rng(seed), (B, heads, top), "ties")
        wd.copy_(dev(w))
        kd.copy_(dev(k))
        g.replay()
        torch.cuda.synchronize()
        want, want_lens = attention.evict_select(w, lens, keep, 4, 20)
        assert np.array_equal(host(kept), want) and np.array_equal(host(kl), want_lens)
        assert_codes_equal(host(kd), attention.compact(k, src, dst, bs, want, want_lens), "k")
