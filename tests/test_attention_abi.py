"""Host-side checks of the attention operators: the C ABI refuses bad arguments before any CUDA work, the binding
refuses bad tensors itself, and the tables of cosines and sines are what their formulas say (no GPU needed)."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def lib(cuda_lib):
    from bit_moe_expert_router_gb300 import attention
    return attention._load()


FAKE = 0x100000  # never dereferenced: every call below is refused, or has no tokens


def _batch(**kw):
    from bit_moe_expert_router_gb300 import attention
    f = dict(n_seqs=4, n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, table_width=3, max_q_len=1, max_kv_len=48,
             dtype=0, k_page_stride=2048, k_row_stride=128, k_head_stride=64, v_page_stride=2048, v_row_stride=128, v_head_stride=64,
             k_cache=FAKE, v_cache=FAKE, block_table=FAKE, q_start=FAKE, kv_len=FAKE)
    f.update(kw)
    return attention._KVBatch(**f)


def _prep(**kw):
    from bit_moe_expert_router_gb300 import attention
    f = dict(cos_sin=FAKE, table_rows=48, rot_dim=64, interleaved=0, q_weight=None, k_weight=None, positions=None, eps=1e-6, weight_offset=0.0)
    f.update(kw)
    return attention._HeadPrep(**f)


def _append(lib, batch, prep, n=4, q=FAKE, qs=(512, 64), k=FAKE, ks=(128, 64), v=FAKE, vs=(128, 64), o=FAKE, os=(512, 64)):
    return lib.moe_w4a8_kv_append(ctypes.byref(batch) if batch else None, ctypes.byref(prep) if prep else None, n, q, *qs, k, *ks, v, *vs,
                                  o, *os, None)


def _attend(lib, batch, n=4, q=FAKE, qs=(512, 64), o=FAKE, os=(512, 64), lse=None, scale=0.125, window=0, ws=FAKE, nbytes=1 << 40):
    return lib.moe_w4a8_paged_attention(ctypes.byref(batch) if batch else None, n, q, *qs, o, *os, lse, scale, window, ws, nbytes, None)


BAD_BATCH = [("n_seqs", 0, 1), ("n_q_heads", 0, 1), ("n_q_heads", 9, 1), ("n_kv_heads", 0, 1), ("head_dim", 0, 1), ("head_dim", 60, 1),
             ("page_size", 0, 1), ("n_pages", 0, 1), ("table_width", 0, 1), ("max_q_len", 0, 1), ("max_kv_len", 0, 1), ("dtype", 2, 1),
             ("dtype", -1, 1), ("k_page_stride", 2044, 1), ("v_row_stride", -8, 1), ("k_cache", None, 1), ("v_cache", FAKE + 8, 1),
             ("block_table", None, 1), ("q_start", FAKE + 2, 1), ("kv_len", None, 1), ("head_dim", 264, 2), ("n_seqs", 2049, 2),
             ("n_q_heads", 2048, 2), ("page_size", 1 << 31, 2), ("n_pages", 1 << 31, 2), ("table_width", 1 << 31, 2)]


@pytest.mark.parametrize("field,value,status", BAD_BATCH)
def test_bad_batches_are_refused(lib, field, value, status):
    b = _batch(**{field: value})
    assert _append(lib, b, _prep(rot_dim=32)) == status
    assert _attend(lib, b) == status


@pytest.mark.parametrize("field,value", [("rot_dim", 63), ("rot_dim", 66), ("rot_dim", -2), ("cos_sin", None), ("cos_sin", FAKE + 4),
                                         ("table_rows", 0), ("q_weight", FAKE + 4), ("k_weight", FAKE + 8), ("positions", FAKE + 2),
                                         ("eps", -1.0), ("eps", math.nan), ("weight_offset", math.inf)])
def test_bad_preps_are_refused(lib, field, value):
    assert _append(lib, _batch(), _prep(**{field: value})) == 1


@pytest.mark.parametrize("kw", [dict(n=-1), dict(q=None), dict(q=FAKE + 2), dict(qs=(516, 64)), dict(ks=(128, -64)), dict(v=None),
                                dict(o=None), dict(os=(512, 4))])
def test_bad_append_rows_are_refused(lib, kw):
    assert _append(lib, _batch(), _prep(), **kw) == 1


@pytest.mark.parametrize("kw,status", [(dict(n=-1), 1), (dict(q=None), 1), (dict(o=FAKE + 2), 1), (dict(os=(512, 60)), 1),
                                       (dict(lse=FAKE + 1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1),
                                       (dict(scale=math.inf), 1), (dict(window=-1), 1), (dict(ws=None), 1), (dict(ws=FAKE + 64), 1),
                                       (dict(nbytes=1 << 10), 3), (dict(n=1 << 28), 2)])
def test_bad_attention_arguments_are_refused(lib, kw, status):
    assert _attend(lib, _batch(), **kw) == status


def test_missing_structs_are_refused(lib):
    assert _append(lib, None, _prep()) == 1
    assert _append(lib, _batch(), None) == 1
    assert _attend(lib, None) == 1
    assert lib.moe_w4a8_paged_attention_workspace_size(None) == 0
    assert lib.moe_w4a8_paged_attention_workspace_size(ctypes.byref(_batch(head_dim=60))) == 0


def test_no_tokens_is_fine(lib):
    assert _append(lib, _batch(), _prep(), n=0, q=None, k=None, v=None, o=None) == 0
    assert _attend(lib, _batch(), n=0, q=None, o=None) == 0


def test_workspace_is_bounded_by_the_gpu_not_by_the_batch(lib):
    sizes = [lib.moe_w4a8_paged_attention_workspace_size(ctypes.byref(_batch(head_dim=d))) for d in (64, 128, 256)]
    assert all(0 < s < 128 << 20 for s in sizes)
    more = lib.moe_w4a8_paged_attention_workspace_size(ctypes.byref(_batch(n_seqs=2048, max_q_len=8192, table_width=4096)))
    assert more == sizes[0]


def test_binding_refuses_wrong_tensors():
    from bit_moe_expert_router_gb300 import attention
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    t, i = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attention.KVBatch(k, k, t, i, i[:2], n_q_heads=4, max_q_len=1)
    with pytest.raises(TypeError, match="dtype"):
        attention.KVBatch(k.float(), k.float(), t, i, i[:2], n_q_heads=4, max_q_len=1)
    with pytest.raises(ValueError, match="CUDA"):
        attention.HeadPrep(torch.zeros(8, 64))
    with pytest.raises(TypeError, match="dtype"):
        attention.HeadPrep(torch.zeros(8, 64, dtype=torch.float64))


def test_rope_table_plain():
    from bit_moe_expert_router_gb300.attention import rope_table
    t = rope_table(50, 12, base=500.0, device="cpu")
    assert t.shape == (50, 12) and t.dtype == torch.float32
    for p in (0, 1, 7, 49):
        for i in range(6):
            a = p * 500.0 ** (-2 * i / 12)
            assert abs(t[p, i].item() - math.cos(a)) < 1e-7
            assert abs(t[p, 6 + i].item() - math.sin(a)) < 1e-7


def test_rope_table_keeps_angles_at_far_positions():
    from bit_moe_expert_router_gb300.attention import rope_table
    t = rope_table(1 << 17, 8, device="cpu")
    p = (1 << 17) - 1
    assert abs(t[p, 0].item() - math.cos(p)) < 1e-7  # the fastest pair: the position itself, in 64 bits


def test_rope_table_scalings():
    from bit_moe_expert_router_gb300.attention import rope_table

    def angles(**kw):  # of position 1: small enough to read back
        t = rope_table(2, 64, device="cpu", **kw).double()
        return torch.atan2(t[1, 32:], t[1, :32]), (t[1, 32:] ** 2 + t[1, :32] ** 2).sqrt()

    plain, one = angles()
    linear, _ = angles(scaling="linear", factor=8.0)
    assert torch.allclose(linear, plain / 8, rtol=1e-5)
    ntk, _ = angles(scaling="ntk", factor=8.0)
    assert abs(ntk[0] - plain[0]) < 1e-6 and abs(ntk[-1] * 8 / plain[-1] - 1) < 1e-3
    yarn, size = angles(scaling="yarn", factor=8.0, original=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.allclose(yarn[turns > 32], plain[turns > 32], rtol=1e-4)
    assert torch.allclose(yarn[turns < 1], plain[turns < 1] / 8, rtol=1e-3)
    assert bool(((yarn >= plain / 8 * 0.999) & (yarn <= plain * 1.001)).all())
    assert torch.allclose(size, torch.full_like(size, 0.1 * math.log(8.0) + 1), rtol=1e-6) and torch.allclose(one, torch.ones_like(one), rtol=1e-6)


@pytest.mark.parametrize("kw", [dict(positions=0), dict(rot_dim=3), dict(rot_dim=0), dict(factor=0.5), dict(scaling="yarn"),
                                dict(scaling="other"), dict(scaling="ntk", rot_dim=2)])
def test_rope_table_refusals(kw):
    from bit_moe_expert_router_gb300.attention import rope_table
    args = dict(positions=4, rot_dim=8, device="cpu")
    args.update(kw)
    with pytest.raises(ValueError):
        rope_table(args.pop("positions"), args.pop("rot_dim"), **args)
