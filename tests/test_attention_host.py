"""The attention and eviction calls on the host: what they refuse, with which
status, before anything reaches a GPU; empty calls; workspace sizes."""

import pytest

import block_scaled_precision_x128_amd as fb
from test_abi_host import FAKE, lib  # noqa: F401  (lib is a fixture)

NULL, ENUM, SHAPE, UNSUPPORTED, WORKSPACE, ALIGN = 1, 2, 3, 4, 5, 7
BIG = 1 << 40


def _attention(lib, **kw):
    a = dict(q=FAKE, q_dt=1, q_tokens=2, heads=8, kv_heads=2, head_dim=128, ld_q=1024, k=FAKE, v=FAKE, num_slots=64,
             table=FAKE, max_blocks=4, block_size=16, batch=2, q_starts=FAKE, kv_lens=FAKE, max_q=1, max_kv=64, fmt=0,
             kind=0, ks=FAKE, vs=FAKE, scale=0.1, out=FAKE, out_dt=1, lse=FAKE, w_in=None, w_out=None, ld_w=0, ws=FAKE,
             ws_bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fp8_kv_attention(*a.values(), None)


def test_kv_attention_refusals(lib):
    for kw in (dict(q_dt=2), dict(out_dt=5), dict(fmt=2), dict(kind=3)):
        assert _attention(lib, **kw) == ENUM, kw
    for kw in (dict(heads=7), dict(kv_heads=0), dict(q_tokens=-1), dict(batch=-1), dict(max_q=-1), dict(max_kv=-1),
               dict(ld_q=1000), dict(num_slots=1 << 31), dict(block_size=0), dict(block_size=(1 << 30) + 1),
               dict(max_kv=65), dict(max_blocks=3), dict(max_kv=(1 << 30) + 1, max_blocks=1 << 40),
               dict(w_out=FAKE, ld_w=63), dict(heads=1 << 40, ld_q=1 << 47), dict(batch=1 << 40),
               dict(q_tokens=1 << 40), dict(max_q=1 << 40), dict(max_blocks=1 << 62, batch=8)):
        assert _attention(lib, **kw) == SHAPE, kw
    for kw in (dict(head_dim=96, ld_q=768), dict(head_dim=0), dict(head_dim=512, ld_q=4096), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attention(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=None), dict(out=None), dict(k=None), dict(v=None), dict(table=None), dict(q_starts=None),
               dict(kv_lens=None), dict(ks=None), dict(vs=None)):
        assert _attention(lib, **kw) == NULL, kw
    for kw in (dict(q=FAKE + 8), dict(ld_q=1028), dict(k=FAKE + 8), dict(v=FAKE + 1), dict(table=FAKE + 4),
               dict(q_starts=FAKE + 4), dict(kv_lens=FAKE + 2), dict(ks=FAKE + 2), dict(vs=FAKE + 1),
               dict(out=FAKE + 4), dict(lse=FAKE + 2), dict(w_out=FAKE + 2, ld_w=64),
               dict(w_out=FAKE, w_in=FAKE + 1, ld_w=64), dict(ws=FAKE + 8)):
        assert _attention(lib, **kw) == ALIGN, kw


def test_kv_attention_workspace(lib):
    size = lib.fp8_kv_attention_workspace_bytes
    # a long cache of one sequence is split; what a call needs is refused below that size
    need = size(1, 32, 8, 128, 1, 1, 1 << 17, 1)
    assert need > 0
    one = dict(q_tokens=1, heads=32, kv_heads=8, ld_q=4096, batch=1, max_blocks=1 << 17, block_size=1, max_kv=1 << 17,
               num_slots=1 << 20, w_out=FAKE, ld_w=1 << 17)
    assert _attention(lib, **one, ws_bytes=need - 1) == WORKSPACE
    assert _attention(lib, **one, ws=None) == WORKSPACE
    for bad in ((1, 32, 7, 128, 1, 1, 64, 0), (1, 32, 8, 100, 1, 1, 64, 0), (-1, 32, 8, 128, 1, 1, 64, 0),
                (1, 32, 8, 128, 1, 1, 1 << 31, 0)):
        assert size(*bad) == 0
    assert fb.fp8_kv_attention_workspace_bytes(1, 32, 8, 128, 1, 1, 1 << 17, True) == need


def test_kv_attention_empty_calls(lib):
    empty = dict(q=None, k=None, v=None, table=None, q_starts=None, kv_lens=None, ks=None, vs=None, out=None, lse=None,
                 ws=None, ws_bytes=0)
    assert _attention(lib, **empty, q_tokens=0) == 0
    assert _attention(lib, **empty, batch=0) == 0
    assert _attention(lib, **empty, heads=0, kv_heads=0, ld_q=0) == 0
    assert _attention(lib, **empty, max_q=0) == 0


def _select(lib, **kw):
    a = dict(w=FAKE, ld_w=64, batch=2, kv_heads=2, kv_lens=FAKE, max_kv=64, keep=16, first=2, recent=4, kept=FAKE,
             kept_lens=FAKE, ws=FAKE, ws_bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fp8_kv_evict_select(*a.values(), None)


def test_evict_select_refusals(lib):
    for kw in (dict(batch=-1), dict(kv_heads=-1), dict(max_kv=-1), dict(keep=-1), dict(first=-1), dict(recent=-1),
               dict(ld_w=63), dict(first=13), dict(recent=15), dict(first=17, recent=0), dict(batch=1 << 40),
               dict(max_kv=1 << 31, ld_w=1 << 31), dict(keep=1 << 31), dict(ld_w=1 << 62)):
        assert _select(lib, **kw) == SHAPE, kw
    for kw in (dict(w=None), dict(kv_lens=None), dict(kept=None), dict(kept_lens=None)):
        assert _select(lib, **kw) == NULL, kw
    for kw in (dict(w=FAKE + 2), dict(kv_lens=FAKE + 4), dict(kept=FAKE + 4), dict(kept_lens=FAKE + 1),
               dict(ws=FAKE + 8)):
        assert _select(lib, **kw) == ALIGN, kw
    need = lib.fp8_kv_evict_select_workspace_bytes(2, 64)
    assert need > 0 and _select(lib, ws_bytes=need - 1) == WORKSPACE and _select(lib, ws=None) == WORKSPACE
    assert lib.fp8_kv_evict_select_workspace_bytes(-1, 64) == 0
    assert _select(lib, batch=0, w=None, kv_lens=None, kept=None, kept_lens=None, ws=None) == 0


def _compact(lib, **kw):
    a = dict(k=FAKE, v=FAKE, num_slots=64, kv_heads=2, head_dim=128, src=FAKE, src_blocks=4, dst=FAKE, dst_blocks=2,
             block_size=16, batch=2, kept=FAKE, kept_lens=FAKE, keep=20, w_in=None, ld_in=0, w_out=None, ld_out=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fp8_kv_compact(*a.values(), None)


def test_compact_refusals(lib):
    for kw in (dict(num_slots=-1), dict(num_slots=1 << 31), dict(head_dim=100), dict(kv_heads=-1), dict(src_blocks=-1),
               dict(dst_blocks=-1), dict(block_size=0), dict(batch=-1), dict(keep=-1), dict(src_blocks=1 << 28),
               dict(dst_blocks=1 << 60), dict(batch=1 << 40), dict(w_in=FAKE, w_out=FAKE, ld_in=64, ld_out=32),
               dict(w_in=FAKE, w_out=FAKE + 64, ld_in=-1)):
        assert _compact(lib, **kw) == SHAPE, kw
    for kw in (dict(k=None), dict(v=None), dict(src=None), dict(dst=None), dict(kept=None), dict(kept_lens=None),
               dict(w_in=FAKE), dict(w_out=FAKE)):
        assert _compact(lib, **kw) == NULL, kw
    for kw in (dict(k=FAKE + 8), dict(v=FAKE + 4), dict(src=FAKE + 4), dict(dst=FAKE + 4), dict(kept=FAKE + 4),
               dict(kept_lens=FAKE + 4), dict(w_in=FAKE + 1, w_out=FAKE, ld_in=64, ld_out=64)):
        assert _compact(lib, **kw) == ALIGN, kw
    none = dict(k=None, v=None, src=None, dst=None, kept=None, kept_lens=None)
    for kw in (dict(batch=0), dict(keep=0), dict(kv_heads=0), dict(head_dim=0)):
        assert _compact(lib, **none, **kw) == 0, kw


def test_compact_refuses_one_table_of_two_widths(lib):
    """One address with rows of two lengths would name two sequences' pages for one."""
    assert _compact(lib, dst=FAKE, src=FAKE, src_blocks=4, dst_blocks=2, batch=2) == SHAPE


def _prompt(lib, **kw):
    a = dict(q=FAKE, ld_q=1024, k=FAKE, ld_k=256, v=FAKE, ld_v=256, tokens=8, heads=8, kv_heads=2, head_dim=128,
             batch=2, starts=FAKE, max_len=8, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.fp8_prompt_attention(*a.values(), None)


def test_prompt_attention_refusals(lib):
    for kw in (dict(heads=7), dict(kv_heads=0), dict(tokens=-1), dict(tokens=1 << 30), dict(batch=-1),
               dict(max_len=-1), dict(ld_q=1016), dict(ld_k=248), dict(ld_v=128), dict(batch=1 << 40),
               dict(heads=1 << 30, ld_q=1 << 40)):
        assert _prompt(lib, **kw) == SHAPE, kw
    for kw in (dict(head_dim=80), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _prompt(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(starts=None), dict(out=None)):
        assert _prompt(lib, **kw) == NULL, kw
    for kw in (dict(q=FAKE + 8), dict(k=FAKE + 2), dict(v=FAKE + 8), dict(out=FAKE + 8), dict(starts=FAKE + 4),
               dict(lse=FAKE + 2), dict(ld_q=1028), dict(ld_k=260), dict(ld_v=258), dict(ws=FAKE + 8)):
        assert _prompt(lib, **kw) == ALIGN, kw
    none = dict(q=None, k=None, v=None, starts=None, out=None, lse=None)
    for kw in (dict(batch=0), dict(tokens=0), dict(max_len=0), dict(heads=0, kv_heads=0)):
        assert _prompt(lib, **none, **kw) == 0, kw


def test_prompt_attention_workspace(lib):
    size = lib.fp8_prompt_attention_workspace_bytes
    assert size(2 * 8192, 32, 8, 128, 2, 8192) == 0             # workgroups enough without a split
    need = size(8192, 1, 1, 128, 1, 8192)
    assert need > 0
    one = dict(tokens=8192, heads=1, kv_heads=1, ld_q=128, ld_k=128, ld_v=128, batch=1, max_len=8192)
    assert _prompt(lib, **one, ws_bytes=need - 1) == WORKSPACE and _prompt(lib, **one, ws=None) == WORKSPACE
    for bad in ((-1, 1, 1, 128, 1, 64), (64, 3, 2, 128, 1, 64), (64, 1, 1, 100, 1, 64), (64, 1, 1, 128, -1, 64)):
        assert size(*bad) == 0


def test_bindings_without_a_gpu_raise():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        fb.fp8_prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int64), 1)
