"""GPU: causal attention of packed prompts against the float64 oracle.

Bound (A = sum_j p_j |v_j|): bf16 inputs have exact products; fp32 sums put a
score off by ds = smax 2^-19 + 2^-22 (1 + |lse|), p by 4 ds, its rounding to
bf16 by 2^-8, the sums over up to 2^12 positions by 2^-16, and out by half a
bf16 step; lse by 2 ds + 2^-18."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x128_amd as fb
import workloads
from gpu_helpers import dev, f32_of_store, host, say
from oracle import attention

pytestmark = pytest.mark.gpu
SENTINEL = 77.25


def _inputs(seed, tokens, H, Hk, D, gain=1.0):
    rng = np.random.default_rng(seed)
    fused = rng.standard_normal((tokens, (H + 2 * Hk) * D)).astype(np.float32)
    fused[:, :H * D] *= gain
    return workloads.f32_to_bf16_bits(fused)


def _split(x, H, Hk, D):
    n = x.shape[0]
    return (x[:, :H * D].reshape(n, H, D), x[:, H * D:(H + Hk) * D].reshape(n, Hk, D),
            x[:, (H + Hk) * D:].reshape(n, Hk, D))


def _run(lens, H, Hk, D, seed=0, gap=0, max_len=None, scale=None, gain=1.0, fused=None, contiguous=False):
    starts = np.concatenate([[gap], gap + np.cumsum(lens)]).astype(np.int64)
    tokens = int(starts[-1]) + gap
    fused = _inputs(seed, tokens, H, Hk, D, gain) if fused is None else fused
    fd = dev(fused)
    q, k, v = (fd[:, :H * D].view(tokens, H, D), fd[:, H * D:(H + Hk) * D].view(tokens, Hk, D),
               fd[:, (H + Hk) * D:].view(tokens, Hk, D))
    if contiguous:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out = torch.full((tokens, H, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tokens, H), SENTINEL, device="cuda")
    top = max(list(lens) + [1]) if max_len is None else max_len
    fb.fp8_prompt_attention(q, k, v, dev(starts), max_len=top, softmax_scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    o, l = f32_of_store(host(out)).astype(np.float64), host(lse).astype(np.float64)
    qn, kn, vn = (f32_of_store(np.ascontiguousarray(x)) for x in _split(fused, H, Hk, D))
    for b, n in enumerate(lens):
        a = int(starts[b])
        w, wl, _, absv, smax = attention.attend(qn[a:a + n], kn[a:a + n], vn[a:a + n], np.arange(n) + 1,
                                                D ** -0.5 if scale is None else scale)
        ds = smax * 2.0 ** -19 + 2.0 ** -22 * (1 + np.abs(wl))
        tol = absv * (4 * ds + 2.0 ** -8 + 2.0 ** -16)[..., None] + np.abs(w) * 2.0 ** -8 + 1e-30
        err = np.abs(o[a:a + n] - w)
        assert (err <= tol).all(), (b, float(np.nanmax(err / tol)), np.argwhere(~(err <= tol))[:4].tolist())
        assert (np.abs(l[a:a + n] - wl) <= 2 * ds + 2.0 ** -18).all(), (b, "lse")
    for x in (out, lse):
        assert (x[:int(starts[0])] == SENTINEL).all() and (x[int(starts[-1]):] == SENTINEL).all()
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2), (7, 1), (6, 6), (33, 1), (16, 2)])
def test_packed_lengths(D, H, Hk):
    say(f"prompt D={D} heads {H}/{Hk}")
    _run([1, 63, 0, 64, 65, 2, 130], H, Hk, D, seed=D + H)


@pytest.mark.parametrize("lens", [[1], [2], [16], [31, 32, 33], [127, 128, 129], [500], [1025, 3]])
def test_lengths(lens):
    say(f"prompt lens={lens}")
    _run(lens, 8, 2, 128, seed=sum(lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,H,Hk", [([1500], 1, 1), ([513, 0, 1100, 2], 3, 1), ([2050], 2, 2), ([4100, 700], 1, 1)])
def test_few_rows_over_many_positions(lens, H, Hk, D):
    """Too few workgroups of rows: the positions are split, in up to nine parts, and joined."""
    say(f"prompt split lens={lens} heads {H}/{Hk} D={D}")
    assert fb.fp8_prompt_attention_workspace_bytes(sum(lens), H, Hk, D, len(lens), max(lens)) > 0
    _run(lens, H, Hk, D, seed=D, gap=2)


def test_a_bound_above_the_lengths_changes_the_split_only():
    a, _ = _run([900, 40], 2, 1, 64, seed=3)
    b, _ = _run([900, 40], 2, 1, 64, seed=3, max_len=5000)
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * a.float().abs().max()


def test_contiguous_inputs_gaps_and_scale():
    _run([40, 100], 4, 4, 64, gap=5, contiguous=True, scale=0.3)
    _run([40, 100], 4, 1, 128, gap=3, max_len=400, scale=1e-3)


def test_large_scores_do_not_overflow():
    _run([300, 70], 4, 2, 64, gain=200.0)


def test_what_lies_outside_a_sequence_has_no_influence():
    """NaN and Inf in the rows between the end of one sequence and the next call's are not read into it."""
    H, Hk, D, lens = 4, 2, 128, [50, 77]
    fused = _inputs(3, 5 + 127 + 5, H, Hk, D)
    fused[:5], fused[132:] = 0x7FC0, 0xFF80
    _run(lens, H, Hk, D, gap=5, fused=fused)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,at", [(3, 1), (64, 63), (200, 130), (1500, 700)])
def test_values_that_are_not_finite(n, at, D):
    """A NaN and an Inf value: tokens in front of it are as without it, tokens that see it get it in that channel."""
    H, Hk = 4, 2
    fused = _inputs(8, n, H, Hk, D)
    starts = dev(np.array([0, n], np.int64))

    def call(x):
        t = dev(x)
        return fb.fp8_prompt_attention(t[:, :H * D].view(n, H, D), t[:, H * D:(H + Hk) * D].view(n, Hk, D),
                                       t[:, (H + Hk) * D:].view(n, Hk, D), starts, max_len=n)

    ref, _ = call(fused)
    bad = fused.copy()
    v0 = (H + Hk) * D
    bad[at, v0 + 9], bad[at, v0 + D + D - 2] = 0xFFC1, 0x7F80       # NaN for kv head 0, Inf for 1
    out, _ = call(bad)
    torch.cuda.synchronize()
    assert torch.equal(out[:at], ref[:at])
    seen, was = out[at:].float(), ref[at:].float()
    assert torch.isnan(seen[:, :2, 9]).all() and (seen[:, 2:, D - 2] == torch.inf).all()
    keep = torch.ones(H, D, dtype=torch.bool)
    keep[:2, 9] = keep[2:, D - 2] = False
    assert torch.equal(seen[:, keep], was[:, keep])
    bad = fused.copy()
    bad[at, H * D + 3] = 0x7FC0                                       # a key of kv head 0
    out, lse = call(bad)
    torch.cuda.synchronize()
    assert torch.equal(out[:at], ref[:at]) and torch.equal(out[:, 2:], ref[:, 2:])
    assert torch.isnan(out[at:, :2].float()).all() and torch.isnan(lse[at:, :2]).all()


def test_nan_of_one_sequence_stays_in_it():
    H, Hk, D = 4, 2, 64
    fused = _inputs(4, 200, H, Hk, D)
    fused[100:] = 0x7FC0
    fd = dev(fused)
    q, k, v = (fd[:, :H * D].view(200, H, D), fd[:, H * D:(H + Hk) * D].view(200, Hk, D), fd[:, (H + Hk) * D:].view(200, Hk, D))
    out, lse = fb.fp8_prompt_attention(q, k, v, dev(np.array([0, 100, 200], np.int64)), max_len=100)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:100].float()).all() and torch.isfinite(lse[:100]).all()
    assert torch.isnan(out[100:].float()).all()


def test_tokens_past_max_len_are_left():
    H, Hk, D = 2, 1, 64
    fd = dev(_inputs(5, 300, H, Hk, D))
    q, k, v = (fd[:, :H * D].view(300, H, D), fd[:, H * D:(H + Hk) * D].view(300, Hk, D), fd[:, (H + Hk) * D:].view(300, Hk, D))
    starts = dev(np.array([0, 290, 300], np.int64))
    whole, _ = fb.fp8_prompt_attention(q, k, v, starts, max_len=290)
    out = torch.full_like(whole, SENTINEL)
    fb.fp8_prompt_attention(q, k, v, starts, max_len=100, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:100], whole[:100]) and torch.equal(out[290:], whole[290:]) and (out[100:290] == SENTINEL).all()


def test_rows_past_two_to_the_31_elements():
    """Row offsets of 32 bits would wrap: the same prompt at both ends of a buffer of 2.5 G elements."""
    H, Hk, D, n, ld, rows = 4, 2, 64, 150, 40960, 61000
    fused = dev(_inputs(9, n, H, Hk, D))
    big = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    out = []
    for a in (0, rows - n):
        big[a:a + n, :(H + 2 * Hk) * D] = fused
        q, k, v = (big[:, x:y].view(rows, -1, D) for x, y in ((0, H * D), (H * D, (H + Hk) * D), ((H + Hk) * D, (H + 2 * Hk) * D)))
        o, lse = fb.fp8_prompt_attention(q, k, v, dev(np.array([a, a + n], np.int64)), max_len=n)
        out.append((o[a:a + n].clone(), lse[a:a + n].clone()))
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    ref, _ = fb.fp8_prompt_attention(fused[:, :H * D].view(n, H, D), fused[:, H * D:(H + Hk) * D].view(n, Hk, D),
                                     fused[:, (H + Hk) * D:].view(n, Hk, D), dev(np.array([0, n], np.int64)), max_len=n)
    torch.cuda.synchronize()
    assert torch.equal(ref, out[0][0])


def test_streams_and_graph():
    H, Hk, D = 8, 2, 128
    fd = dev(_inputs(6, 260, H, Hk, D))
    q, k, v = (fd[:, :H * D].view(260, H, D), fd[:, H * D:(H + Hk) * D].view(260, Hk, D), fd[:, (H + Hk) * D:].view(260, Hk, D))
    starts = dev(np.array([0, 200, 260], np.int64))
    ref, ref_lse = fb.fp8_prompt_attention(q, k, v, starts, max_len=200)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, lse = fb.fp8_prompt_attention(q, k, v, starts, max_len=200, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out2, lse2 = torch.empty_like(ref), torch.empty_like(ref_lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fb.fp8_prompt_attention(q, k, v, starts, max_len=200, out=out2, lse=lse2)
    for _ in range(3):
        out2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, ref) and torch.equal(lse2, ref_lse)


def test_binding_refuses():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.tensor([0, 4], device="cuda")
    with pytest.raises(TypeError):
        fb.fp8_prompt_attention(x.float(), x, x, s, 4)
    with pytest.raises(TypeError):
        fb.fp8_prompt_attention(x, x, x, s.int(), 4)
    with pytest.raises(ValueError):
        fb.fp8_prompt_attention(x, x[:2], x, s, 4)
    with pytest.raises(ValueError):
        fb.fp8_prompt_attention(x, x, x, s.cpu(), 4)
    with pytest.raises(ValueError):
        fb.fp8_prompt_attention(x, x.transpose(0, 1).contiguous().transpose(0, 1), x, s, 4)
    y = torch.zeros(4, 2, 96, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fb.Fp8Error):
        fb.fp8_prompt_attention(y, y, y, s, 4)
