"""The paged K/V cache's calls refuse bad arguments on the host, before any
launch (no CUDA call is reached on these paths)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def kvs():
    from kv_index_scan_b200 import build
    build.build()
    import kv_index_scan_b200
    return kv_index_scan_b200


def _kv(kvs, **change):
    f = dict(K=4096, V=4096, page_stride=2 * 16 * 128, head_stride=16 * 128, token_stride=128, table=4096, table_ld=8,
             n=4096, R=2, G=2, D=128, page=16, max_pages=8, num_pages=32)
    f.update(change)
    return kvs.PagedKVC(*f.values())


BAD_CACHES = [(dict(K=None), 1), (dict(V=None), 1), (dict(table=None), 1), (dict(n=None), 1), (dict(D=64), 2),
              (dict(R=0), 1), (dict(G=0), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2),
              (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(table_ld=7), 1), (dict(token_stride=100), 1),
              (dict(token_stride=132), 1), (dict(head_stride=-128), 1), (dict(page_stride=0), 1), (dict(K=4104), 1),
              (dict(max_pages=1 << 27, table_ld=1 << 27), 2), (dict(R=1 << 14, G=1 << 12), 2)]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_descriptor_checks(kvs, change, status):
    L, kv = kvs._lib, _kv(kvs, **change)
    ref = ctypes.pointer(kv)
    assert L.kvs_paged_append(ref, 4096, 4096, 1 << 20, None, kv.R, None, None, None, None, None) == status
    d = kvs.PagedDecodeArgsC(ref, 4096, 0, 4, 0, 0, 1.0, 4096, None, None, None)
    assert L.paged_decode_attn(ctypes.byref(d), 4096, 1 << 40, None, None) == status
    p = kvs.PagedPromptArgsC(ref, 4096, 1 << 20, 4096, 4, 4, 0, 0, 1.0, 4096, 1 << 20, None)
    assert L.paged_prompt_attn(ctypes.byref(p), 4096, 1 << 40, None, None) == status
    e = kvs.PagedEvictArgsC(ref, 4096, None, None, 8, 0, 0, 4096, None, 4096, 4096)
    assert L.kvs_paged_evict(ctypes.byref(e), 4096, 1 << 40, None, None) == status
    assert L.kvs_last_error()


def test_null_descriptors(kvs):
    L = kvs._lib
    assert L.kvs_paged_append(None, 4096, 4096, 256, None, 2, None, None, None, None, None) == kvs.KVS_EINVAL
    assert L.paged_decode_attn(None, None, 0, None, None) == kvs.KVS_EINVAL
    assert L.paged_prompt_attn(None, None, 0, None, None) == kvs.KVS_EINVAL
    assert L.kvs_paged_evict(None, None, 0, None, None) == kvs.KVS_EINVAL


@pytest.mark.parametrize("args,word", [
    ((None, 4096, 256, None, 2, None, None, None), b"non-null"),
    ((4096, 4096, 256, None, 3, None, None, None), b"one token a request"),
    ((4096, 4096, 256, 4096, -1, None, None, None), b"T=-1"),
    ((4096, 4096, 128, None, 2, None, None, None), b"new_ld"),
    ((4096, 4096, 260, None, 2, None, None, None), b"new_ld"),
    ((4104, 4096, 256, None, 2, None, None, None), b"aligned"),
    ((4096, 4096, 256, None, 2, None, None, 4096), b"seen"),
])
def test_append_checks(kvs, args, word):
    kv = _kv(kvs)
    K, V, ld, cu, T, mass, pos, seen = args
    st = kvs._lib.kvs_paged_append(ctypes.pointer(kv), K, V, ld, cu, T, mass, pos, seen, None, None)
    assert st == kvs.KVS_EINVAL and word in kvs._lib.kvs_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(q_dtype=2), 1), (dict(H=0), 1), (dict(H=9), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(mass=4096), 1), (dict(mass_out=4096), 1), (dict(q=4100), 1),
    (dict(out=4100), 1)])
def test_decode_checks(kvs, change, status):
    kv = _kv(kvs)
    f = dict(kv=ctypes.pointer(kv), q=4096, q_dtype=0, H=4, window=0, sinks=0, scale=1.0, out=4096, lse=None,
             mass=None, mass_out=None)
    f.update(change)
    a = kvs.PagedDecodeArgsC(*f.values())
    assert kvs._lib.paged_decode_attn(ctypes.byref(a), 4096, 1 << 40, None, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(H=9), 1),
    (dict(window=-1), 1), (dict(sinks=-5), 1), (dict(scale=float("inf")), 1), (dict(q_ld=1020), 1), (dict(q_ld=512), 1), (dict(out_ld=1028), 1),
    (dict(q=4104), 1), (dict(out=4104), 1), (dict(T=1 << 30), 2)])
def test_prompt_checks(kvs, change, status):
    kv = _kv(kvs)
    f = dict(kv=ctypes.pointer(kv), q=4096, q_ld=1024, cu=4096, T=4, H=4, window=0, sinks=0, scale=1.0, out=4096,
             out_ld=1024, lse=None)
    f.update(change)
    a = kvs.PagedPromptArgsC(*f.values())
    assert kvs._lib.paged_prompt_attn(ctypes.byref(a), 4096, 1 << 40, None, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(mass=None), 1), (dict(mass_out=None), 1), (dict(n_out=None), 1), (dict(src=None), 1), (dict(pos=4096), 1),
    (dict(pos_out=4096), 1), (dict(budget=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1),
    (dict(sinks=5, recent=4), 1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1)])
def test_evict_checks(kvs, change, status):
    kv = _kv(kvs)
    f = dict(kv=ctypes.pointer(kv), mass=4096, pos=None, seen=None, budget=8, sinks=0, recent=0, mass_out=4096,
             pos_out=None, n_out=4096, src=4096)
    f.update(change)
    a = kvs.PagedEvictArgsC(*f.values())
    assert kvs._lib.kvs_paged_evict(ctypes.byref(a), 4096, 1 << 40, None, None) == status


def test_workspace_checks(kvs):
    kv = _kv(kvs)
    a = kvs.PagedEvictArgsC(ctypes.pointer(kv), 4096, None, None, 8, 0, 0, 4096, None, 4096, 4096)
    need = kvs._lib.kvs_paged_evict_workspace_size(2, 2, 8)
    assert need > 0
    assert kvs._lib.kvs_paged_evict(ctypes.byref(a), None, 0, None, None) == kvs.KVS_EWORKSPACE
    assert kvs._lib.kvs_paged_evict(ctypes.byref(a), 4096, need - 1, None, None) == kvs.KVS_EWORKSPACE
    assert kvs._lib.kvs_paged_evict(ctypes.byref(a), 4104, 1 << 40, None, None) == kvs.KVS_EINVAL


def test_prompt_workspace(kvs):
    """Few queries over a long cache are split and need a workspace; many do not."""
    kv = _kv(kvs, max_pages=4096, table_ld=4096)
    need = kvs._lib.kvs_paged_prompt_workspace_size(2, 2, 4, 8, 65536, 0, 0)
    assert need > 0 and kvs._lib.kvs_paged_prompt_workspace_size(2, 2, 4, 1 << 16, 65536, 0, 0) == 0
    assert kvs._lib.kvs_paged_prompt_workspace_size(2, 2, 4, 8, 128, 0, 0) == 0
    assert kvs._lib.kvs_paged_prompt_workspace_size(2, 2, 4, 8, 65536, 200, 4) == 0  # a short window
    a = kvs.PagedPromptArgsC(ctypes.pointer(kv), 4096, 1024, 4096, 8, 4, 0, 0, 1.0, 4096, 1024, None)
    for ws, size, status in ((None, 0, kvs.KVS_EWORKSPACE), (4096, need - 1, kvs.KVS_EWORKSPACE), (4104, need, kvs.KVS_EINVAL)):
        assert kvs._lib.paged_prompt_attn(ctypes.byref(a), ws, size, None, None) == status


def test_binding_refuses_host_tensors(kvs):
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvs.PagedKV(pool, pool, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_pages"):
        kvs.PagedKV(pool.float(), pool, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_decode_timeout_selftest_checks(kvs):
    """The failure-path self-test refuses bad arguments before any launch."""
    kv = _kv(kvs)
    f = dict(kv=ctypes.pointer(kv), q=4096, q_dtype=1, H=4, window=0, sinks=0, scale=1.0, out=4096, lse=None,
             mass=None, mass_out=None)
    def call(warp=0, cycles=10 ** 6, status=4096, ws=1 << 40, **change):
        a = kvs.PagedDecodeArgsC(*{**f, **change}.values())
        return kvs._lib.kvs_selftest_paged_decode_timeout(ctypes.byref(a), 4096, ws, warp, cycles, status, None)
    for bad in (dict(warp=-1), dict(warp=5), dict(cycles=999), dict(cycles=3 * 10 ** 9), dict(status=None), dict(q=None),
                dict(H=9)):
        assert call(**bad) == kvs.KVS_EINVAL, bad
    assert call(q_dtype=0) == kvs.KVS_EUNSUPPORTED and call(mass=4096, mass_out=4096) == kvs.KVS_EUNSUPPORTED
    assert call(ws=0) == kvs.KVS_EWORKSPACE


def test_prompt_timeout_selftest_checks(kvs):
    kv = _kv(kvs)
    f = dict(kv=ctypes.pointer(kv), q=4096, q_ld=1024, cu=4096, T=4, H=4, window=0, sinks=0, scale=1.0, out=4096,
             out_ld=1024, lse=None)
    def call(warp=0, cycles=10 ** 6, status=4096, **change):
        a = kvs.PagedPromptArgsC(*{**f, **change}.values())
        return kvs._lib.kvs_selftest_paged_prompt_timeout(ctypes.byref(a), warp, cycles, status, None)
    for bad in (dict(warp=-1), dict(warp=12), dict(cycles=999), dict(cycles=3 * 10 ** 9), dict(status=None), dict(T=0),
                dict(out=None)):
        assert call(**bad) == kvs.KVS_EINVAL, bad


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.4e38, float("inf"), float("-inf"), float("nan"), 0.0])
def test_scales_without_a_finite_base_2_form_are_refused(kvs, scale):
    """The kernels multiply by scale * log2(e): where that is not finite a logit of 0 would become NaN."""
    kv = _kv(kvs)
    d = kvs.PagedDecodeArgsC(ctypes.pointer(kv), 4096, 0, 4, 0, 0, scale, 4096, None, None, None)
    assert kvs._lib.paged_decode_attn(ctypes.byref(d), 4096, 1 << 40, None, None) == kvs.KVS_EINVAL
    assert b"scale" in kvs._lib.kvs_last_error()
    p = kvs.PagedPromptArgsC(ctypes.pointer(kv), 4096, 1024, 4096, 4, 4, 0, 0, scale, 4096, 1024, None)
    assert kvs._lib.paged_prompt_attn(ctypes.byref(p), 4096, 1 << 40, None, None) == kvs.KVS_EINVAL
    assert b"scale" in kvs._lib.kvs_last_error()


@pytest.mark.parametrize("R,G,H,T,cap,window,sinks", [
    (1, 1, 4, 700, 65536, 0, 0), (2, 2, 4, 900, 65536, 0, 0), (40, 8, 8, 500, 131072, 0, 0), (3, 8, 1, 3000, 30000, 0, 0),
    (1, 8, 5, 2500, 200000, 9000, 300), (64, 1, 3, 400, 16384, 0, 0), (2, 2, 4, 900, 128, 0, 0), (1, 4, 4, 1, 65536, 0, 0)])
def test_prompt_workspace_bound(kvs, R, G, H, T, cap, window, sinks):
    """A workspace of the bound is enough for every call of up to T queries, and one of them needs all of it; the
    size of a call itself falls to 0 where queries are many."""
    size = kvs._lib.kvs_paged_prompt_workspace_size
    bound = kvs._lib.kvs_paged_prompt_workspace_bound(R, G, H, T, cap, window, sinks)
    assert bound == max(size(R, G, H, t, cap, window, sinks) for t in range(1, T + 1))
    assert bound >= kvs._lib.kvs_paged_prompt_workspace_bound(R, G, H, max(1, T // 3), cap, window, sinks)


def test_prompt_workspace_bound_of_many_queries(kvs):
    """Beyond the last split call more queries change nothing; sizes that no call takes ask for nothing."""
    bound = kvs._lib.kvs_paged_prompt_workspace_bound
    assert kvs._lib.kvs_paged_prompt_workspace_size(1, 8, 4, 1 << 20, 65536, 0, 0) == 0
    assert bound(1, 8, 4, 1 << 20, 65536, 0, 0) == bound(1, 8, 4, 1 << 16, 65536, 0, 0) > 0
    for bad in ((0, 8, 4, 9, 65536, 0, 0), (1, 0, 4, 9, 65536, 0, 0), (1, 8, 0, 9, 65536, 0, 0), (1, 8, 9, 9, 65536, 0, 0),
                (1, 8, 4, 0, 65536, 0, 0)):
        assert bound(*bad) == 0


@pytest.mark.parametrize("budget", [(1 << 30) + 1, 2 ** 31 - 1])
def test_evict_budgets_beyond_any_cache_are_refused(kvs, budget):
    """Slots are counted in 32 bits, and a block's steps beyond the last: a budget near 2^31 would wrap."""
    kv = _kv(kvs)
    a = kvs.PagedEvictArgsC(ctypes.pointer(kv), 4096, None, None, budget, 0, 0, 4096, None, 4096, 4096)
    assert kvs._lib.kvs_paged_evict(ctypes.byref(a), None, 0, None, None) == kvs.KVS_EUNSUPPORTED
    assert b"budget" in kvs._lib.kvs_last_error()
