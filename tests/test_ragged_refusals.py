"""Refusals of the ragged-batch entry points: every one happens on the host, before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import krea2_inputs as KI

FAKE = 1 << 20


@pytest.fixture(scope="module")
def K2():
    from flow_matching_stream_b200 import build
    build.build()
    import flow_matching_stream_b200 as K2
    return K2


def batch(**kw):
    from flow_matching_stream_b200 import _lib
    s = _lib.Krea2PagedBatch()
    v = dict(R=2, M=10, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=4, page_size=16, num_pages=9, k_pages=FAKE,
             v_pages=FAKE)
    v.update(kw)
    for k, x in v.items():
        setattr(s, k, x)
    return s


BAD_BATCHES = [(dict(R=0), -1), (dict(M=0), -1), (dict(M=(1 << 30) + 1), -1), (dict(R=4097), -5), (dict(max_pages=0), -1),
               (dict(page_size=0), -1), (dict(page_size=24), -5), (dict(num_pages=0), -1),
               (dict(max_pages=1 << 20, page_size=1 << 12), -1), (dict(q_start=None), -1), (dict(kv_len=None), -1),
               (dict(page_table=None), -1), (dict(k_pages=None), -1), (dict(v_pages=None), -1),
               (dict(k_pages=FAKE + 8), -1), (dict(v_pages=FAKE + 2), -1)]


@pytest.mark.parametrize("change,code", BAD_BATCHES)
def test_bad_batches(K2, change, code):
    lib, d = K2.lib(), K2.dims_struct(KI.FULL)
    b = batch(**change)
    assert lib.krea2_paged_kv_append(ctypes.byref(d), ctypes.byref(b), 0, FAKE, FAKE, FAKE, FAKE, None) == code
    assert lib.krea2_gqa_attention_paged(ctypes.byref(d), ctypes.byref(b), 0, 0, FAKE, FAKE, FAKE, FAKE, None, None, FAKE,
                                         FAKE, 1 << 40, None) == code


def test_bad_attention_arguments(K2):
    lib, d, b = K2.lib(), K2.dims_struct(KI.FULL), batch()
    need = lib.krea2_paged_attention_workspace_size(ctypes.byref(d), ctypes.byref(b), 0)

    def call(T=0, dtype=0, qkvg=FAKE, qw=FAKE, cos=FAKE, sin=FAKE, mask=None, end=None, out=FAKE, ws=FAKE, n=need):
        return lib.krea2_gqa_attention_paged(ctypes.byref(d), ctypes.byref(b), T, dtype, qkvg, qw, cos, sin, mask, end,
                                             out, ws, n, None)

    assert call(T=-1) == -1 and call(dtype=2) == -1
    for name in ("qkvg", "qw", "cos", "sin", "out"):
        assert call(**{name: None}) == -1
    for name in ("qkvg", "out", "qw", "cos", "sin"):
        assert call(**{name: FAKE + 8}) == -1
    if need:
        assert call(ws=None) == -2 and call(ws=FAKE + 128) == -2 and call(n=need - 1) == -2
    assert lib.krea2_gqa_attention_paged(ctypes.byref(d), None, 0, 0, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE,
                                         need, None) == -1
    assert lib.krea2_paged_attention_workspace_size(ctypes.byref(d), ctypes.byref(batch(R=0)), 0) == 0
    assert lib.krea2_paged_kv_append(ctypes.byref(d), ctypes.byref(b), 0, None, FAKE, FAKE, FAKE, None) == -1
    for i in range(4):
        at = [FAKE + 8 if i == k else FAKE for k in range(4)]
        assert lib.krea2_paged_kv_append(ctypes.byref(d), ctypes.byref(b), 0, *at, None) == -1
    bad = K2.dims_struct(KI.FULL)
    bad.axes[0] = 30
    assert lib.krea2_paged_kv_append(ctypes.byref(bad), ctypes.byref(b), 0, FAKE, FAKE, FAKE, FAKE, None) == -1


GOOD = dict(q_start=[0, 3, 3, 8], kv_len=[20, 0, 5], page_table=[[4, 1, -1], [-1, -1, -1], [2, 9, 7]], num_pages=5,
            page_size=16, rows=10)


def test_batch_check(K2):
    K2.paged_batch_check(**GOOD)
    for change in (dict(q_start=[1, 3, 3, 8]), dict(q_start=[0, 5, 3, 8]), dict(q_start=[0, 3, 3, 11]),
                   dict(q_start=[0, -1, 3, 8]), dict(kv_len=[2, 0, 5]), dict(kv_len=[49, 0, 5]), dict(kv_len=[20, -1, 5]),
                   dict(kv_len=[33, 0, 5]), dict(kv_len=[20, 0, 17]), dict(num_pages=4),
                   dict(page_table=[[4, 2, -1], [-1, -1, -1], [2, 9, 7]]),  # both append to rows of page 2
                   dict(page_table=[[4, 1, -1], [-1, -1, -1], [-3, 9, 7]])):
        with pytest.raises(K2.Krea2Error) as e:
            K2.paged_batch_check(**{**GOOD, **change})
        assert e.value.code == -1, change
    # a prefix that is only read may be shared, slots of one page that differ may both be appended to
    K2.paged_batch_check([0, 1, 2], [17, 18], [[3, 1], [3, 0]], 5, 16, 2)
    K2.paged_batch_check([0, 1, 2], [17, 18], [[3, 1], [3, 1]], 5, 16, 2)
    with pytest.raises(ValueError):
        K2.paged_batch_check([0, 1], [17, 18], [[3, 1], [3, 0]], 5, 16, 2)


def test_bad_lora_arguments(K2):
    from flow_matching_stream_b200 import _lib
    lib = K2.lib()

    def call(dtype=0, epi=0, M=10, N=256, K=128, R=2, n_ad=1, rank=16, A=FAKE, W=FAKE, out=FAKE, gate=None, rpb=0,
             stride=0, ws=FAKE, n=1 << 30, **ptr):
        s = _lib.Krea2Lora()
        s.R, s.n_adapters, s.rank = R, n_ad, rank
        for k in ("row_start", "adapter", "scale", "down", "up"):
            setattr(s, k, ptr.get(k, FAKE))
        return lib.krea2_lora_linear(dtype, epi, M, N, K, A, W, ctypes.byref(s), out, gate, rpb, stride, ws, n, None)

    for kw, code in ((dict(dtype=3), -1), (dict(epi=5), -1), (dict(M=0), -1), (dict(K=-64), -1), (dict(R=0), -1),
                     (dict(R=5000), -5), (dict(M=(1 << 22) + 1), -5), (dict(rank=0), -5), (dict(rank=12), -5),
                     (dict(rank=264), -5), (dict(N=200), -5), (dict(K=100), -5), (dict(epi=1, N=192, dtype=1), -1),
                     (dict(n_ad=0), -1), (dict(A=None), -1), (dict(W=None), -1), (dict(out=None), -1),
                     (dict(row_start=None), -1), (dict(adapter=None), -1), (dict(scale=None), -1), (dict(down=None), -1),
                     (dict(up=None), -1), (dict(A=FAKE + 8), -1), (dict(up=FAKE + 2), -1), (dict(down=FAKE + 8), -1),
                     (dict(epi=2), -1), (dict(epi=2, gate=FAKE, rpb=-1), -1), (dict(epi=2, gate=FAKE, stride=-1), -1),
                     (dict(ws=None), -2), (dict(ws=FAKE + 16), -2), (dict(n=16), -2)):
        assert call(**kw) == code, kw
    assert lib.krea2_lora_linear(0, 0, 8, 128, 64, FAKE, FAKE, None, FAKE, None, 0, 0, FAKE, 1 << 30, None) == -1
    assert lib.krea2_lora_workspace_size(0, 0, 8, 100, 64, 1, 16) == 0
    assert lib.krea2_lora_workspace_size(0, 0, 8, 128, 64, 1, 16) > 0


def test_binding_checks_tensors(K2):
    t = torch.zeros
    i32 = torch.int32
    with pytest.raises(ValueError):  # CPU tensors
        K2.PagedBatch(t(3, dtype=i32), t(2, dtype=i32), t(2, 4, dtype=i32), t(9, 16, 128), t(9, 16, 128), 10)
    with pytest.raises(TypeError):
        K2.PagedBatch(t(3), t(2, dtype=i32), t(2, 4, dtype=i32), t(9, 16, 128), t(9, 16, 128), 10)
    with pytest.raises(ValueError):
        K2.PagedBatch(t(2, dtype=i32), t(2, dtype=i32), t(2, 4, dtype=i32), t(9, 16, 128), t(9, 16, 128), 10)
    with pytest.raises(ValueError):
        K2.LoraAdapters(t(2, 16, 64), t(2, 128, 8), t(2))
    with pytest.raises(TypeError):
        K2.LoraAdapters(t(2, 16, 64), t(2, 128, 16), t(2, dtype=torch.float64))


def test_rows_per_batch_that_does_not_fit_32_bits(K2):
    # its low 32 bits are 0, which would read a gate row per request where the caller's gate has one row
    import types

    from flow_matching_stream_b200 import _lib
    t, bf = torch.zeros, torch.bfloat16
    adapters = types.SimpleNamespace(dev=0, dtype=bf, K=64, Nw=128, rank=16, struct=_lib.Krea2Lora())
    for rows_per_batch in (2 ** 32, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="rows_per_batch"):
            K2.lora_linear(K2.KREA2_EPI_RESID, t(10, 64, dtype=bf), t(128, 64, dtype=bf), adapters,
                           t(4, dtype=torch.int32), t(3, dtype=torch.int32), t(10, 128), t(1 << 16, dtype=torch.uint8),
                           gate=t(1, 128), rows_per_batch=rows_per_batch)


def test_batch_check_of_values_that_do_not_fit(K2):
    # lengths, page numbers and sizes are refused, never cut to 32 bits or to whole numbers
    big = 2 ** 32
    for change in (dict(q_start=np.array([0, 3, 3, 8 + big])), dict(kv_len=torch.tensor([20, big, 5])),
                   dict(kv_len=[20 - big, 0, 5]), dict(page_table=np.array([[4 + big, 1, -1], [-1] * 3, [2, 9, 7]])),
                   dict(rows=10 + big), dict(num_pages=5 + big), dict(page_size=16 - big)):
        with pytest.raises(ValueError, match="32 bits"):
            K2.paged_batch_check(**{**GOOD, **change})
    for change in (dict(kv_len=[20.9, 0, 5]), dict(q_start=torch.tensor([0.0, 3, 3, 8])),
                   dict(page_table=[["4", "1", "2"]] * 3)):
        with pytest.raises(TypeError):
            K2.paged_batch_check(**{**GOOD, **change})
    for dt in (np.int64, np.uint8, np.int32):  # other integer types of fitting values are fine
        K2.paged_batch_check(**{**GOOD, "kv_len": np.array(GOOD["kv_len"], dtype=dt)})


def test_binding_refuses_sizes_that_do_not_fit(K2):
    import types

    from flow_matching_stream_b200 import _lib
    t, i32, big = torch.zeros, torch.int32, 2 ** 32
    lengths = (t(3, dtype=i32), t(2, dtype=i32))
    pages = (t(9, 16, 128), t(9, 16, 128))
    with pytest.raises(ValueError, match="rows.*32 bits"):
        K2.PagedBatch(*lengths, t(2, 4, dtype=i32), *pages, big + 10)
    with pytest.raises(ValueError, match="max_pages.*32 bits"):
        K2.PagedBatch(*lengths, t(2, 1, dtype=i32).expand(2, big + 4), *pages, 10)
    batch = types.SimpleNamespace(dev=0, rows=10, R=2, kv_cols=KI.FULL.KVD, dtype=torch.float32)
    with pytest.raises(ValueError, match="text_mask.*32 bits"):
        K2.gqa_attention_paged(KI.FULL, batch, t(1), t(1), t(1), t(1), t(2, 1, dtype=torch.uint8).expand(2, big + 8),
                               None, t(1), None)
    sizes = dict(epilogue=0, M=10, Nw=256, K=128, R=2, rank=16)
    assert K2.lora_workspace_size(torch.float32, **sizes) > 0
    for name in sizes:
        with pytest.raises(ValueError, match=f"{name}.*32 bits"):
            K2.lora_workspace_size(torch.float32, **{**sizes, name: sizes[name] + big})
    with pytest.raises(ValueError, match="K.*32 bits"):
        K2.LoraAdapters(t(1, 1, 1).expand(2, 16, big + 64), t(2, 128, 16), t(2))
    adapters = types.SimpleNamespace(dev=0, dtype=torch.float32, K=1, Nw=128, rank=16, struct=_lib.Krea2Lora())
    call = (t(128, 1), adapters, t(3, dtype=i32), t(2, dtype=i32), t(1), t(1))
    with pytest.raises(ValueError, match="M.*32 bits"):
        K2.lora_linear(0, t(1, 1).expand(big + 1, 1), *call)
    with pytest.raises(ValueError, match="epilogue.*32 bits"):
        K2.lora_linear(big + 1, t(10, 1), *call)


def test_too_many_fp32_rows_are_refused_before_a_launch(K2):
    from flow_matching_stream_b200 import _lib
    lib, s = K2.lib(), _lib.Krea2Lora()
    s.R, s.n_adapters, s.rank = 2, 1, 16
    for k in ("row_start", "adapter", "scale", "down", "up"):
        setattr(s, k, FAKE)
    before = lib.krea2_launch_count()
    assert lib.krea2_lora_linear(1, 0, 1 << 22, 2048, 64, FAKE, FAKE, ctypes.byref(s), FAKE, None, 0, 0, FAKE, 1 << 40,
                                 None) == -5
    assert lib.krea2_launch_count() == before
