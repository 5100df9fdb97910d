"""GPU parity of the paged key/value append and the paged attention against fp64."""
import pytest
import torch

import krea2_inputs as KI
from ragged_ref import Ragged, off

pytestmark = pytest.mark.gpu

# Root mean square of one rounding to bf16 relative to the value: at most half a step, 2^-8, over sqrt(3).
BF16_RMS = 2.0 ** -8 / 3 ** 0.5
# Attention in bf16 rounds q_hat, the probabilities and the output; each moves the result by at most one
# rounding's RMS of its size (scores q.k/sqrt(D) of normalised q and k move by about one rounding of
# a unit value). A single element is off by half a step of its own, 2^-8, and by the errors of the probabilities,
# two roundings relative to sum_k p_k |v_k| (not to the element, which may cancel), within 8 deviations.
TOL_ATTN_BF16 = 3 * BF16_RMS
# fp32: D-term dot products (RMS sqrt(D) 2^-24 of a unit score) and sums over the keys.
TOL_ATTN_F32 = 1e-5

D64 = KI.Dims(C=512, H=8, Hkv=2, D=64, F=512, axes=(16, 24, 24))


def dims(H, Hkv):
    return KI.Dims(C=H * 128, H=H, Hkv=Hkv, D=128, F=1024, axes=(32, 48, 48))


@pytest.fixture(scope="module")
def K2(cuda_device):
    import flow_matching_stream_b200 as K2
    return K2


def batch_of(K2, b):
    return K2.PagedBatch(b.q_start, b.kv_len, b.table, b.k_pages, b.v_pages, b.rows)


def run_attention(K2, b, text_mask=None, key_end=None, fill=7.0, ws=None):
    pb = batch_of(K2, b)
    out = torch.full((b.rows, b.d.HD), fill, device="cuda", dtype=b.dtype)
    if ws is None:
        n = K2.paged_attention_workspace_size(b.d, pb, b.dtype)
        ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    K2.gqa_attention_paged(b.d, pb, b.qkvg, b.qw, b.cos, b.sin, text_mask, key_end, out, ws)
    K2.check_device_error()
    return out


def compare(b, out, ref, size, rows=None):
    """Rows of requests (or `rows` of them) against fp64, and zeros where a token has no readable key."""
    rows = slice(0, b.start[-1]) if rows is None else rows
    out, ref, size = out[rows].double(), ref[rows], size[rows]
    rel, _ = off(out, ref)
    if b.dtype == torch.bfloat16:
        assert rel <= TOL_ATTN_BF16
        assert bool(((out - ref).abs() <= 2.0 ** -8 * ref.abs() + 16 * BF16_RMS * size).all())
    else:
        assert rel <= TOL_ATTN_F32
        assert bool(((out - ref).abs() <= 8 * TOL_ATTN_F32 * size).all())


def check_attention(K2, b, text_mask=None, key_end=None):
    out = run_attention(K2, b, text_mask, key_end)
    compare(b, out, *b.attention(text_mask, key_end))
    assert torch.all(out[b.start[-1]:] == 7.0)  # rows behind the last request
    return out


def causal(b):
    end = [b.kv[r] - b.new[r] + i + 1 for r in range(b.R) for i in range(b.new[r])]
    return torch.tensor(end + [0] * (b.rows - b.start[-1]), dtype=torch.int32, device="cuda")


def random_mask(b, T, keep, seed=3):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(b.R, T, generator=g) < keep).to(torch.uint8).cuda()


# ------------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("d", [dims(8, 2), D64, KI.FULL], ids=["d128", "d64", "full"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new,kv,page", [
    ([1], [1], 16), ([5, 0, 1, 33], [5, 40, 64, 97], 16), ([70, 1, 129], [70, 128, 200], 64), ([3, 200], [50, 248], 48)])
def test_append(K2, d, dtype, new, kv, page):
    b = Ragged(d, new, kv, page, dtype, "cuda", spare=3)
    k0, v0 = b.k_pages.clone(), b.v_pages.clone()
    kr, vr = b.appended()
    K2.paged_kv_append(d, batch_of(K2, b), b.qkvg, b.kw, b.cos, b.sin)
    K2.check_device_error()
    assert torch.equal(b.v_pages, vr.to(dtype))
    written = torch.zeros(k0.shape[:2], dtype=torch.bool, device="cuda")
    for r in range(b.R):
        p, s = b.slots(r)
        if b.new[r]:
            written[p[-b.new[r]:], s[-b.new[r]:]] = True
    assert torch.equal(b.k_pages[~written], k0[~written]) and torch.equal(b.v_pages[~written], v0[~written])
    rel, big = off(b.k_pages[written], kr[written])
    # one rounding of the output; in fp32 a handful of roundings of 2^-24 each, within 16 of them
    tol = 2.0 ** -8 if dtype == torch.bfloat16 else 16 * 2.0 ** -24
    assert big <= tol * 1.01


# --------------------------------------------------------------------------------------- attention

SHAPES = [
    ([1], [1], 16), ([1], [77], 16), ([1, 1, 1], [64, 65, 63], 64), ([2, 0, 31, 33], [2, 9, 200, 128], 16),
    ([128, 1], [128, 1000], 32), ([129, 64, 3], [321, 64, 700], 128), ([40], [300], 48), ([5, 7], [8200, 4100], 64)]


@pytest.mark.parametrize("new,kv,page", SHAPES)
@pytest.mark.parametrize("d", [dims(8, 2), dims(6, 3), dims(3, 3)], ids=["g4", "g2", "g1"])
def test_attention_bf16(K2, d, new, kv, page):
    b = Ragged(d, new, kv, page, torch.bfloat16, "cuda", spare=5)
    b.poison()
    check_attention(K2, b)
    check_attention(K2, b, key_end=causal(b))
    check_attention(K2, b, text_mask=random_mask(b, 70, 0.5))


@pytest.mark.parametrize("new,kv,page", SHAPES)
@pytest.mark.parametrize("d,dtype", [(D64, torch.float32), (D64, torch.bfloat16), (dims(6, 2), torch.bfloat16),
                                     (dims(4, 1), torch.float32)], ids=["d64f32", "d64bf16", "g3", "d128f32"])
def test_attention_simt(K2, d, dtype, new, kv, page):
    b = Ragged(d, new, kv, page, dtype, "cuda", spare=5)
    b.poison()
    check_attention(K2, b)
    check_attention(K2, b, text_mask=random_mask(b, 70, 0.5), key_end=causal(b))


def test_attention_full_heads_long(K2):
    b = Ragged(KI.FULL, [300, 1, 64], [5000, 20001, 2049], 64, torch.bfloat16, "cuda", spare=1)
    b.poison()
    check_attention(K2, b, text_mask=random_mask(b, 512, 0.3))


def test_attention_whole_rounds(K2):
    # more items (64 tokens of a KV head) than CTAs: whole items in turn, the rest in equal shares
    b = Ragged(KI.FULL, [900, 70], [1000, 300], 64, torch.bfloat16, "cuda")
    b.poison()
    check_attention(K2, b)
    check_attention(K2, b, key_end=causal(b))


def test_attention_short_tables_are_not_cut(K2):
    # tables of at most 256 keys: items are handed out whole
    b = Ragged(dims(8, 2), [190] * 38 + [1, 0, 77], [190] * 38 + [192, 3, 77], 64, torch.bfloat16, "cuda", spare=2)
    b.poison()
    check_attention(K2, b, key_end=causal(b))
    few = Ragged(dims(8, 2), [1] * 90, [1 + (7 * r) % 180 for r in range(90)], 64, torch.bfloat16, "cuda")
    few.poison()
    check_attention(K2, few)


@pytest.mark.parametrize("keep", [0.0, 0.02, 0.9])
def test_attention_masks(K2, keep):
    # keep 0: requests shorter than the mask have no readable key at all and output zeros
    b = Ragged(dims(8, 2), [3, 40, 1, 130], [64, 200, 500, 150], 16, torch.bfloat16, "cuda")
    mask = random_mask(b, 200, keep)
    for key_end in (None, causal(b)):
        out = check_attention(K2, b, mask, key_end)
        empty = b.attention(mask, key_end)[1].amax(1) == 0
        assert (keep > 0) or bool(empty.any())
        assert torch.all(out[empty] == 0)


def test_attention_masked_keys_may_hold_anything(K2):
    # NaN and infinities in keys that the mask removes, and behind the last key, change nothing
    d = dims(8, 2)
    for value in (float("nan"), float("inf"), -float("inf")):
        b = Ragged(d, [40, 1], [300, 131], 16, torch.bfloat16, "cuda")
        mask = random_mask(b, 150, 0.6)
        want = run_attention(K2, b, mask)
        b.poison(value)
        for r in range(b.R):
            p, s = b.slots(r)
            gone = ~mask[r, :b.kv[r]].bool()
            t = torch.nonzero(gone).flatten()
            b.k_pages[p[t], s[t]] = value
            b.v_pages[p[t], s[t]] = value
        assert torch.equal(run_attention(K2, b, mask), want)


@pytest.mark.parametrize("few", [False, True])
def test_attention_key_ends_of_any_order(K2, few):
    # values below a token's own position are raised to it, values past the last key cut to it, in any order
    new, kv = ([1, 2, 1], [300, 700, 64]) if few else ([70, 3, 200], [300, 700, 220])
    b = Ragged(dims(8, 2), new, kv, 16, torch.bfloat16, "cuda", spare=4)
    g = torch.Generator().manual_seed(4)
    end = torch.randint(-5, 900, (b.rows,), generator=g, dtype=torch.int32)
    end[::7], end[3::7] = 0, 2 ** 31 - 1
    check_attention(K2, b, key_end=end.cuda())
    check_attention(K2, b, text_mask=random_mask(b, 250, 0.4), key_end=end.cuda())


@pytest.mark.parametrize("new", [[1], [90]])
def test_attention_long_sparse_masks(K2, new):
    # more masked tiles than one word of the kernel's tile bits, and a mask longer than a request
    b = Ragged(dims(8, 2), new + [2], [4000, 150], 64, torch.bfloat16, "cuda")
    b.poison()
    mask = torch.zeros(2, 3001, dtype=torch.uint8, device="cuda")
    mask[0, [5, 1000, 1001, 2047, 2048, 2900]] = 1
    mask[1, 70:149] = 1
    check_attention(K2, b, text_mask=mask)
    mask[0] = 0  # the first request sees only the keys behind the mask
    check_attention(K2, b, text_mask=mask)


@pytest.mark.parametrize("new", [[1, 1, 1], [100, 33, 3]])
def test_attention_nan_token_stays_alone(K2, new):
    b = Ragged(dims(8, 2), new, [400, 100, 300], 16, torch.bfloat16, "cuda")
    want = run_attention(K2, b)
    row = b.start[1]
    b.qkvg[row, :b.d.HD] = float("nan")
    got = run_attention(K2, b)
    keep = torch.arange(b.rows, device="cuda") != row
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[row]).all()


@pytest.mark.parametrize("d,dtype", [(dims(8, 2), torch.bfloat16), (D64, torch.float32)])
def test_empty_batches(K2, d, dtype):
    # no request has a new token: nothing is written
    b = Ragged(d, [0, 0, 0], [0, 70, 16], 16, dtype, "cuda", spare=40)
    k0 = b.k_pages.clone()
    K2.paged_kv_append(d, batch_of(K2, b), b.qkvg, b.kw, b.cos, b.sin)
    out = run_attention(K2, b)
    assert torch.all(out == 7.0) and torch.equal(b.k_pages, k0)


def test_attention_many_requests(K2):
    # more requests than a block has threads, most of them empty
    n = [1 if r % 5 == 0 else (3 if r % 41 == 0 else 0) for r in range(1500)]
    kv = [max(n[r], (r * 37) % 200) for r in range(1500)]
    b = Ragged(dims(4, 1), n, kv, 16, torch.bfloat16, "cuda", spare=2)
    b.poison()
    K2.paged_kv_append(b.d, batch_of(K2, b), b.qkvg, b.kw, b.cos, b.sin)
    check_attention(K2, b)


@pytest.mark.parametrize("d,dtype,page", [(dims(8, 2), torch.bfloat16, 64), (D64, torch.float32, 16)])
def test_offsets_past_32_bits(K2, d, dtype, page):
    # a pool of more than 2^31 elements; the requests' pages lie at its end
    b = Ragged(d, [1, 40], [200, 130], page, dtype, "cuda")
    pages = 2 ** 31 // (page * d.KVD) + b.num_pages + 1
    kp, vp = (torch.empty(pages, page, d.KVD, device="cuda", dtype=dtype) for _ in range(2))
    first = pages - b.num_pages
    kp[first:], vp[first:] = b.k_pages, b.v_pages
    b.table = torch.where(b.table >= 0, b.table + first, b.table)
    b.k_pages, b.v_pages, b.num_pages = kp, vp, pages
    pb = batch_of(K2, b)
    K2.paged_kv_append(d, pb, b.qkvg, b.kw, b.cos, b.sin)
    check_attention(K2, b)
    for r in range(b.R):
        p, s = b.slots(r)
        want = b.qkvg[b.rowsof(r), d.HD + d.KVD:d.HD + 2 * d.KVD]
        assert torch.equal(vp[p[-b.new[r]:], s[-b.new[r]:]], want)


def test_attention_shared_prefix_pages(K2):
    # two requests whose first pages are the same ones
    b = Ragged(dims(8, 2), [3, 9], [140, 150], 16, torch.bfloat16, "cuda")
    b.table[1, :8] = b.table[0, :8]
    check_attention(K2, b)


def test_attention_large_scores(K2):
    # q and k far from unit size: one key dominates, other exponentials underflow
    d = dims(8, 2)
    b = Ragged(d, [70], [400], 16, torch.bfloat16, "cuda")
    b.qw += 4.0
    b.k_pages *= 8.0
    out = run_attention(K2, b)
    ref, _ = b.attention()
    assert torch.isfinite(out).all()
    # scores reach several hundred: a rounding of q_hat (2^-8) moves them by more than 1, so only tokens
    # whose largest score leads by a wide margin are comparable
    x = b.qkvg[:, :d.HD].reshape(70, d.H, d.D)
    from ragged_ref import norm_rope
    q = norm_rope(x, b.qw, b.cos, b.sin, d.eps)
    p, s = b.slots(0)
    k = b.k_pages[p, s].double().reshape(400, d.Hkv, d.D)
    clear = torch.zeros(70, d.H, dtype=torch.bool, device="cuda")
    for h in range(d.H):
        z = q[:, h] @ k[:, h // 4].T / d.D ** 0.5
        top = z.topk(2, 1).values
        # worst case of the rounding of q_hat: 2^-8 sum |q_i k_i| / sqrt(D) for each of the two keys
        move = 2.0 ** -8 * (q[:, h].abs() @ k[:, h // 4].abs().T / d.D ** 0.5).amax(1)
        clear[:, h] = top[:, 0] - top[:, 1] > 2 * move + 8
    assert int(clear.sum()) > 10
    e = (out.double() - ref).reshape(70, d.H, d.D)[clear]
    assert float(e.abs().max()) <= (2.0 ** -8 + 2 * 400 * 2.0 ** -11) * float(ref.abs().max())


def test_attention_matches_the_contiguous_cache(K2):
    # one request, pages in order: the paged attention answers what the contiguous cache's does
    d = KI.FULL
    P, Nq, T = 300, 256, 128
    L = P + Nq
    b = Ragged(d, [Nq], [L], 64, torch.bfloat16, "cuda")
    mask = random_mask(b, T, 0.7)
    cap = b.max_pages * 64
    kc, vc = (torch.zeros(1, cap, d.KVD, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    p, s = b.slots(0)
    K2.paged_kv_append(d, batch_of(K2, b), b.qkvg, b.kw, b.cos, b.sin)
    kc[0, :L], vc[0, :L] = b.k_pages[p, s], b.v_pages[p, s]
    kc2, vc2 = kc.clone(), vc.clone()
    K2.kv_cache_append(d, 1, Nq, P, b.qkvg, b.kw, b.cos, b.sin, kc2, vc2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    want = torch.empty(Nq, d.HD, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(K2.kv_cache_attention_workspace_size(d, 1, Nq, torch.bfloat16), dtype=torch.uint8, device="cuda")
    K2.gqa_attention_kv_cache(d, 1, T, L, Nq, b.qkvg, b.qw, b.cos, b.sin, mask, kc, vc, None, want, ws)
    got = run_attention(K2, b, mask)
    # both differ from fp64 by at most TOL_ATTN_BF16 in the 2-norm
    rel, _ = off(got, want)
    assert rel <= 2 * TOL_ATTN_BF16


def test_attention_captured_with_changing_lengths(K2):
    # one graph serves batches of other lengths, pages and row counts
    d = dims(8, 2)
    cases = [([64, 1, 3], [300, 1000, 3]), ([1, 1, 1], [77, 64, 1500]), ([0, 66, 2], [40, 66, 130])]
    bs = [Ragged(d, n, k, 16, torch.bfloat16, "cuda", seed=i) for i, (n, k) in enumerate(cases)]
    rows, pages, width = 70, max(b.num_pages for b in bs), max(b.max_pages for b in bs)
    z = torch.zeros
    q_start, kv_len = z(4, dtype=torch.int32, device="cuda"), z(3, dtype=torch.int32, device="cuda")
    table = z(3, width, dtype=torch.int32, device="cuda")
    kp, vp = (z(pages, 16, d.KVD, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    qkvg = z(rows, d.qkvg_cols, device="cuda", dtype=torch.bfloat16)
    cos, sin = z(rows, 64, device="cuda"), z(rows, 64, device="cuda")
    out = z(rows, d.HD, device="cuda", dtype=torch.bfloat16)
    pb = K2.PagedBatch(q_start, kv_len, table, kp, vp, rows)
    ws = torch.empty(max(256, K2.paged_attention_workspace_size(d, pb, torch.bfloat16)), dtype=torch.uint8,
                     device="cuda")
    qw, kw = bs[0].qw, bs[0].kw

    def step():
        K2.paged_kv_append(d, pb, qkvg, kw, cos, sin)
        K2.gqa_attention_paged(d, pb, qkvg, qw, cos, sin, None, None, out, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for b in bs:
        b.qw, b.kw = qw, kw
        n = b.rows
        q_start.copy_(b.q_start), kv_len.copy_(b.kv_len)
        table[:, :b.max_pages] = b.table
        kp[:b.num_pages], vp[:b.num_pages] = b.k_pages, b.v_pages
        qkvg[:n], cos[:n], sin[:n] = b.qkvg, b.cos, b.sin
        out.fill_(7.0)
        graph.replay()
        K2.check_device_error()
        b.k_pages, b.v_pages = kp[:b.num_pages], vp[:b.num_pages]
        compare(b, out, *b.attention())
        assert torch.all(out[n:] == 7.0)


def test_attention_repeats_bit_for_bit_and_on_two_streams(K2):
    d = dims(8, 2)
    a = Ragged(d, [1, 1, 40], [5000, 300, 1000], 16, torch.bfloat16, "cuda", seed=1)
    b = Ragged(d, [130, 1], [130, 4000], 64, torch.bfloat16, "cuda", seed=2)
    want = [run_attention(K2, x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pbs = [batch_of(K2, x) for x in (a, b)]
    outs = [torch.zeros(x.rows, d.HD, device="cuda", dtype=torch.bfloat16) for x in (a, b)]
    wss = [torch.empty(max(256, K2.paged_attention_workspace_size(d, p, torch.bfloat16)), dtype=torch.uint8,
                       device="cuda") for p in pbs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, p, o, w, s in zip((a, b), pbs, outs, wss, streams):
            K2.gqa_attention_paged(d, p, x.qkvg, x.qw, x.cos, x.sin, None, None, o, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_inconsistent_batches_are_reported_and_skipped(K2):
    # the host check refuses these batches (test_ragged_refusals.py); the kernels' own checks keep every
    # access inside the arrays, skip the request and report it
    d = dims(8, 2)
    good = Ragged(d, [3, 40, 2], [64, 200, 500], 16, torch.bfloat16, "cuda")
    ref, size = good.attention()
    for field, index, value in (("kv_len", 1, 39), ("kv_len", 1, 10 ** 6), ("kv_len", 1, -5), ("q_start", 1, 90),
                                ("q_start", 2, -1), ("q_start", 3, 10 ** 6)):
        b = Ragged(d, [3, 40, 2], [64, 200, 500], 16, torch.bfloat16, "cuda")
        getattr(b, field)[index] = value
        pb = batch_of(K2, b)
        k0 = b.k_pages.clone()
        out = torch.full((b.rows, d.HD), 7.0, device="cuda", dtype=torch.bfloat16)
        ws = torch.empty(max(256, K2.paged_attention_workspace_size(d, pb, torch.bfloat16)), dtype=torch.uint8,
                         device="cuda")
        K2.gqa_attention_paged(d, pb, b.qkvg, b.qw, b.cos, b.sin, None, None, out, ws)
        with pytest.raises(K2.Krea2Error) as e:
            K2.check_device_error()
        assert e.value.code == -1
        if field == "kv_len":  # the other requests are answered, the inconsistent one's rows stay
            # (not bit for bit: where long requests are cut depends on the whole batch's work)
            compare(good, out, ref, size, slice(0, 3))
            compare(good, out, ref, size, slice(43, 45))
            assert torch.all(out[3:43] == 7.0)
        K2.paged_kv_append(d, pb, b.qkvg, b.kw, b.cos, b.sin)
        with pytest.raises(K2.Krea2Error):
            K2.check_device_error()
        if field == "kv_len":
            p, s = good.slots(1)
            assert torch.equal(b.k_pages[p, s], k0[p, s])
    K2.check_device_error()


@pytest.mark.parametrize("page", [-1, 10 ** 6])
def test_page_numbers_outside_the_pool_are_reported(K2, page):
    d = dims(8, 2)
    good = Ragged(d, [3, 40], [64, 200], 16, torch.bfloat16, "cuda")
    want = run_attention(K2, good)
    b = Ragged(d, [3, 40], [64, 200], 16, torch.bfloat16, "cuda")
    b.table[1, 2] = page
    pb = batch_of(K2, b)
    out = torch.zeros(b.rows, d.HD, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(max(256, K2.paged_attention_workspace_size(d, pb, torch.bfloat16)), dtype=torch.uint8,
                     device="cuda")
    K2.gqa_attention_paged(d, pb, b.qkvg, b.qw, b.cos, b.sin, None, None, out, ws)
    with pytest.raises(K2.Krea2Error) as e:
        K2.check_device_error()
    assert e.value.code == -1
    assert torch.equal(out[:3], want[:3])


# ----------------------------------------------- batches of about one new token per request (16 query rows an item)

@pytest.mark.parametrize("d", [dims(8, 2), dims(6, 3), dims(3, 3)], ids=["g4", "g2", "g1"])
def test_attention_few_rows(K2, d):
    b = Ragged(d, [1, 0, 2, 1, 3], [300, 50, 1700, 64, 5000], 16, torch.bfloat16, "cuda", spare=1)
    assert b.rows <= 2 * b.R
    b.poison()
    g = torch.Generator().manual_seed(6)
    end = torch.randint(-5, 6000, (b.rows,), generator=g, dtype=torch.int32).cuda()
    for mask in (None, random_mask(b, 250, 0.4)):
        for key_end in (None, end, causal(b)):
            check_attention(K2, b, mask, key_end)


def test_attention_one_long_chunk_among_empty_requests(K2):
    # 16-row items by the row count, yet one request has all the rows: whole rounds of items and a rest
    b = Ragged(dims(8, 2), [0] * 300 + [1400] + [0] * 420, [3] * 300 + [1500] + [0] * 420, 64, torch.bfloat16, "cuda",
               spare=11)
    assert b.rows <= 2 * b.R and 1400 // 4 * b.d.Hkv > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    b.poison()
    check_attention(K2, b)
    check_attention(K2, b, key_end=causal(b))


def test_attention_causal_prompts(K2):
    # prompts read from nothing: most of an item's key tiles lie behind its tokens' key ends
    for new in ([1500], [400, 1, 650, 64]):
        b = Ragged(dims(8, 2), new, new, 64, torch.bfloat16, "cuda", spare=3)
        b.poison()
        check_attention(K2, b, key_end=causal(b))
