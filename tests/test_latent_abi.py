"""Host-side checks of latent attention: the C ABI refuses bad arguments before any CUDA work, and the binding refuses bad
tensors itself (no GPU needed)."""
import ctypes
import math

import pytest
import torch

FAKE = 0x100000  # never dereferenced: every call below is refused, or has no tokens


@pytest.fixture(scope="module")
def lib(cuda_lib):
    from bit_moe_expert_router_gb300 import latent
    return latent._load()


def _batch(**kw):
    from bit_moe_expert_router_gb300 import latent
    f = dict(n_seqs=4, n_heads=8, latent_dim=128, rot_dim=64, page_size=24, n_pages=10, table_width=2, max_q_len=1, max_kv_len=48, dtype=0,
             page_stride=24 * 192, row_stride=192, cache=FAKE, block_table=FAKE, q_start=FAKE, kv_len=FAKE)
    f.update(kw)
    return latent._LatentBatch(**f)


def _prep(**kw):
    from bit_moe_expert_router_gb300 import attention
    f = dict(cos_sin=FAKE, table_rows=48, rot_dim=64, interleaved=0, q_weight=None, k_weight=None, positions=None, eps=1e-6, weight_offset=0.0)
    f.update(kw)
    return attention._HeadPrep(**f)


def _append(lib, batch, prep, n=4, c=FAKE, cs=192, k=FAKE, ks=192, q=FAKE, qs=(1536, 192), o=FAKE, os=(1536, 192)):
    return lib.moe_w4a8_latent_append(ctypes.byref(batch) if batch else None, ctypes.byref(prep) if prep else None, n, c, cs, k, ks, q, *qs, o, *os, None)


def _attend(lib, batch, n=4, q=FAKE, qs=(1536, 192), o=FAKE, os=(1024, 128), lse=None, scale=0.125, ws=FAKE, nbytes=1 << 40):
    return lib.moe_w4a8_latent_attention(ctypes.byref(batch) if batch else None, n, q, *qs, o, *os, lse, scale, ws, nbytes, None)


BAD_BATCH = [("n_seqs", 0, 1), ("n_heads", 0, 1), ("latent_dim", 0, 1), ("latent_dim", 100, 1), ("rot_dim", -8, 1), ("rot_dim", 60, 1), ("page_size", 0, 1),
             ("n_pages", 0, 1), ("table_width", 0, 1), ("max_q_len", 0, 1), ("max_kv_len", 0, 1), ("dtype", 2, 1), ("dtype", -1, 1),
             ("page_stride", 4612, 1), ("page_stride", 0, 1), ("row_stride", -8, 1), ("row_stride", 184, 1), ("cache", None, 1), ("cache", FAKE + 8, 1),
             ("block_table", None, 1), ("q_start", FAKE + 2, 1), ("kv_len", None, 1), ("latent_dim", 520, 2), ("rot_dim", 72, 2), ("n_seqs", 2049, 2),
             ("n_heads", 1025, 2), ("page_size", 12, 2), ("page_size", 1 << 31, 2), ("n_pages", 1 << 31, 2), ("table_width", 1 << 31, 2),
             ("page_stride", 1 << 39, 2), ("row_stride", 1 << 39, 2)]


@pytest.mark.parametrize("field,value,status", BAD_BATCH)
def test_bad_batches_are_refused(lib, field, value, status):
    b = _batch(**{field: value})
    assert _append(lib, b, _prep(rot_dim=b.rot_dim)) == status
    assert _attend(lib, b) == status
    if field not in ("cache", "block_table", "q_start", "kv_len"):
        assert lib.moe_w4a8_latent_attention_workspace_size(ctypes.byref(b)) == 0


@pytest.mark.parametrize("kw", [dict(rot_dim=32), dict(cos_sin=None), dict(cos_sin=FAKE + 4), dict(table_rows=0), dict(q_weight=FAKE), dict(k_weight=FAKE + 8),
                                dict(positions=FAKE + 2), dict(eps=-1.0), dict(eps=math.nan), dict(weight_offset=math.inf)])
def test_bad_preps_are_refused(lib, kw):
    assert _append(lib, _batch(), _prep(**kw)) == 1


@pytest.mark.parametrize("kw", [dict(c=None), dict(c=FAKE + 4), dict(cs=-8), dict(cs=196), dict(k=None), dict(ks=4), dict(q=None), dict(qs=(1536, 4)), dict(qs=(-8, 192)),
                                dict(o=None), dict(o=FAKE + 2), dict(os=(1536, 190)), dict(n=-1)])
def test_bad_append_arguments_are_refused(lib, kw):
    assert _append(lib, _batch(), _prep(), **kw) == 1


@pytest.mark.parametrize("kw,status", [(dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(qs=(1536, 4)), 1), (dict(o=None), 1), (dict(os=(-8, 128)), 1), (dict(lse=FAKE + 2), 1),
                                       (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(ws=None), 1),
                                       (dict(ws=FAKE + 16), 1), (dict(n=-1), 1), (dict(nbytes=1 << 16), 3), (dict(n=1 << 29), 2), (dict(n=(1 << 28) - 60), 2)])
def test_bad_attend_arguments_are_refused(lib, kw, status):
    assert _attend(lib, _batch(), **kw) == status


def test_nothing_to_do_and_null_structs(lib):
    assert _append(lib, None, _prep()) == 1 and _append(lib, _batch(), None) == 1 and _attend(lib, None) == 1
    assert lib.moe_w4a8_latent_attention_workspace_size(None) == 0
    # no tokens: the token arrays are not looked at
    assert _append(lib, _batch(), _prep(), n=0, c=None, k=None, q=None, o=None) == 0
    assert _attend(lib, _batch(), n=0, q=None, o=None) == 0
    # a single page has no stride
    assert _attend(lib, _batch(n_pages=1, page_stride=0), n=0) == 0


def test_the_workspace_does_not_go_by_the_tokens(lib):
    size = lib.moe_w4a8_latent_attention_workspace_size
    small, large = _batch(), _batch(n_seqs=2000, n_heads=128, max_q_len=8192, max_kv_len=1 << 20)
    assert size(ctypes.byref(small)) == size(ctypes.byref(large)) > 0


def test_the_binding_refuses(lib):
    from bit_moe_expert_router_gb300 import latent
    i32 = dict(dtype=torch.int32)
    cache, table, start, lens = torch.zeros(4, 16, 192, dtype=torch.bfloat16), torch.zeros(2, 2, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32)
    for error, match, c in ((TypeError, "dtype", cache.float()), (ValueError, "CUDA", cache)):
        with pytest.raises(error, match=match):
            latent.LatentBatch(c, table, start, lens, n_heads=4, latent_dim=128, max_q_len=1)


def test_the_package_offers_them():
    import bit_moe_expert_router_gb300 as moe
    for name in ("moe_w4a8_latent_append", "moe_w4a8_latent_attention", "LatentBatch", "moe_w4a8_route_scored", "RouteRule", "moe_w4a8_forward_bf16_routed"):
        assert name in moe.__all__ and getattr(moe, name)
