"""GPU parity of the projection with per-request adapters against fp64."""
import pytest
import torch

from ragged_ref import lora_ref, off

pytestmark = pytest.mark.gpu

# One rounding of the output to bf16 has an RMS of at most 2^-8 / sqrt(3) of the value, and 2^-8 at most.
# The low-rank product keeps 16 bits and the accumulators fp32, which add below a tenth of that.
TOL_BF16 = 1.1 * 2.0 ** -8 / 3 ** 0.5
# fp32 results of K-term sums: roundings of 2^-24 of the running sum, RMS sqrt(K) of them at most
# (K = 16384: 128 * 6e-8 = 7.6e-6), for the shared product and for the low-rank one.
TOL_F32 = 1.6e-5


@pytest.fixture(scope="module")
def K2(cuda_device):
    import flow_matching_stream_b200 as K2
    return K2


class Case:
    def __init__(self, K2, epilogue, rows, K, N, rank, n_ad, dtype, ids=None, spare=0, seed=0, rows_per_batch=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, scale=1.0, dt=dtype):
            return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

        self.K2, self.epilogue, self.rank, self.rows_per_batch = K2, epilogue, rank, rows_per_batch
        self.start = [0]
        for n in rows:
            self.start.append(self.start[-1] + n)
        self.M, self.R, self.used = self.start[-1] + spare, len(rows), self.start[-1]
        self.ids = [i % n_ad for i in range(self.R)] if ids is None else ids
        self.A, self.W = rnd(self.M, K), rnd(N, K, scale=K ** -0.5)
        self.down, self.up = rnd(n_ad, rank, K, scale=K ** -0.5), rnd(n_ad, N, rank, scale=0.7 * rank ** -0.5)
        self.scale = torch.rand(n_ad, device="cuda", generator=g) + 0.5
        self.row_start = torch.tensor(self.start, dtype=torch.int32, device="cuda")
        self.adapter = torch.tensor(self.ids, dtype=torch.int32, device="cuda")
        gates = self.R if rows_per_batch == 0 else -(-self.M // rows_per_batch)
        self.gate = rnd(gates, N, scale=0.5, dt=torch.float32) if epilogue == "resid" else None
        cols = N // 2 if epilogue == "swiglu" else N
        self.out0 = rnd(self.M, cols, dt=torch.float32 if epilogue == "resid" else dtype)
        self.epi = {"store": K2.KREA2_EPI_STORE, "swiglu": K2.KREA2_EPI_SWIGLU, "resid": K2.KREA2_EPI_RESID}[epilogue]
        self.lora = K2.LoraAdapters(self.down, self.up, self.scale)
        n = K2.lora_workspace_size(dtype, self.epi, self.M, N, K, self.R, rank)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere

    def run(self, stream=None):
        out = self.out0.clone()
        self.K2.lora_linear(self.epi, self.A, self.W, self.lora, self.row_start, self.adapter, out, self.ws,
                            gate=self.gate, rows_per_batch=self.rows_per_batch, stream=stream)
        return out

    def ref(self):
        return lora_ref(self.A, self.W, self.down, self.up, self.scale, self.start, self.ids, self.epilogue, self.out0,
                        self.gate, self.rows_per_batch)

    def check(self):
        out = self.run()
        self.K2.check_device_error()
        tol = TOL_BF16 if out.dtype == torch.bfloat16 else TOL_F32
        rel, big = off(out[:self.used], self.ref()[:self.used])
        assert rel <= tol and big <= 8 * tol
        assert torch.equal(out[self.used:], self.out0[self.used:])
        return out


@pytest.mark.parametrize("epilogue", ["store", "swiglu", "resid"])
@pytest.mark.parametrize("rows,rank,ids,spare", [
    ([1], 8, None, 0), ([1], 16, [-1], 3), ([1, 1, 1, 1, 1], 16, None, 0), ([128], 64, None, 0),
    ([100, 0, 28, 1], 24, [0, 1, -1, 2], 0), ([3, 130, 127, 60, 7], 40, None, 29), ([300, 5], 128, None, 200),
    ([64] * 9, 256, None, 1), ([1] * 67, 32, None, 0), ([31, 33, 200], 72, [2, 0, 2], 130)])
def test_lora_bf16(K2, epilogue, rows, rank, ids, spare):
    Case(K2, epilogue, rows, 640, 768, rank, 3, torch.bfloat16, ids=ids, spare=spare).check()


@pytest.mark.parametrize("epilogue", ["store", "swiglu", "resid"])
@pytest.mark.parametrize("rows,K,N,rank,spare", [([1], 256, 640, 8, 0), ([64, 8, 1], 256, 640, 8, 2),
                                                 ([5, 0, 70], 72, 128, 40, 0), ([129, 1], 100, 384, 256, 70)])
def test_lora_f32(K2, epilogue, rows, K, N, rank, spare):
    Case(K2, epilogue, rows, K, N, rank, 2, torch.float32, ids=[1, -1, 0][:len(rows)], spare=spare).check()


@pytest.mark.parametrize("epilogue,rows,K,N,rank", [
    ("store", [1, 301, 37, 1024, 1, 128, 77, 1], 6144, 15360, 64), ("store", [7], 6144, 6144, 16),
    ("swiglu", [600, 1, 555], 6144, 32768, 16), ("resid", [1152, 1101, 1029, 30], 16384, 6144, 32),
    ("resid", [3, 1], 6144, 6144, 8)])
def test_lora_model_sizes(K2, epilogue, rows, K, N, rank):
    Case(K2, epilogue, rows, K, N, rank, 4, torch.bfloat16, ids=[0, 3, -1, 1, 2, 0, 3, 1][:len(rows)], spare=9).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_residual_gate_by_rows(K2, dtype):
    # rows_per_batch > 0: the gate row goes by the packed row, as krea2_linear's does
    Case(K2, "resid", [50, 30, 70], 128, 256, 16, 3, dtype, spare=10, rows_per_batch=40).check()


def test_lora_without_adapters_is_linear(K2):
    # the sums may run in another order than linear's; each of the two is within TOL_BF16 of the exact product
    c = Case(K2, "store", [200, 3, 96], 1024, 1536, 16, 2, torch.bfloat16, ids=[-1, -1, -1])
    want = torch.empty_like(c.out0)
    K2.linear(c.epi, c.A, c.W, want)
    rel, big = off(c.run(), want)
    assert rel <= 2 * TOL_BF16 and big <= 16 * TOL_BF16


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("epilogue", ["store", "swiglu", "resid"])
def test_lora_empty_batch(K2, epilogue, dtype):
    c = Case(K2, epilogue, [0, 0], 128, 256, 16, 2, dtype, spare=300)
    assert torch.equal(c.run(), c.out0)
    c.K2.check_device_error()


def test_lora_many_requests(K2):
    rows = [1 if r % 3 == 0 else (2 if r % 50 == 0 else 0) for r in range(900)]
    Case(K2, "store", rows, 256, 256, 8, 5, torch.bfloat16, ids=[(r * 7) % 6 - 1 for r in range(900)], spare=3).check()


def test_lora_infinite_low_rank_product(K2):
    # down overflows for one request: its rows are infinite (or NaN where infinities cancel), others are not touched
    c = Case(K2, "store", [10, 10], 128, 128, 8, 2, torch.bfloat16)
    want = c.run()
    c.A[10:] = 1.0
    c.down[1] = 0.0
    c.down[1, 0] = 3e38
    c.up[1] = 1.0
    got = c.run()
    assert torch.equal(got[:10], want[:10])
    assert torch.all(got[10:] == float("inf"))


def test_lora_other_rows_do_not_matter(K2):
    # a row's result depends on its own values only: NaN in another request's rows of the same tile stays there
    c = Case(K2, "store", [20, 20, 20], 256, 256, 16, 3, torch.bfloat16)
    want = c.run()
    c.A[20:40] = float("nan")
    got = c.run()
    assert torch.equal(got[:20], want[:20]) and torch.equal(got[40:], want[40:])
    assert torch.isnan(got[20:40]).all()


def test_lora_repeats_bit_for_bit_captured_and_on_two_streams(K2):
    a = Case(K2, "store", [1, 70, 200], 1024, 1536, 48, 3, torch.bfloat16, seed=1)
    b = Case(K2, "resid", [33, 129], 512, 768, 16, 2, torch.bfloat16, seed=2)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for c, s, w in zip((a, b), streams, want):
            with torch.cuda.stream(s):
                out = c.run(stream=s)
            s.synchronize()
            assert torch.equal(out, w)
    # captured: row starts and adapters change between replays
    out = torch.zeros_like(a.out0)

    def step():
        K2.lora_linear(a.epi, a.A, a.W, a.lora, a.row_start, a.adapter, out, a.ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for start, ids in (([0, 1, 71, 271], [0, 1, 2]), ([0, 100, 100, 150], [2, 0, -1]), ([0, 0, 0, 1], [0, 0, 1])):
        a.start, a.ids, a.used = start, ids, start[-1]
        a.row_start.copy_(torch.tensor(start, dtype=torch.int32))
        a.adapter.copy_(torch.tensor(ids, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        K2.check_device_error()
        rel, big = off(out[:a.used], a.ref()[:a.used])
        assert rel <= TOL_BF16 and big <= 8 * TOL_BF16
        assert torch.all(out[a.used:] == 7.0)


def test_lora_inconsistent_arrays_are_reported(K2):
    for field, index, value in (("adapter", 1, 3), ("adapter", 1, -2), ("row_start", 1, 90), ("row_start", 3, 10 ** 6),
                                ("row_start", 2, -1), ("row_start", 0, 5)):
        c = Case(K2, "store", [20, 40, 9], 256, 256, 16, 3, torch.bfloat16)
        want = c.run()
        K2.check_device_error()
        getattr(c, field)[index] = value
        got = c.run()
        with pytest.raises(K2.Krea2Error) as e:
            K2.check_device_error()
        assert e.value.code == -1
        if field == "adapter":
            assert torch.equal(got[:20], want[:20]) and torch.equal(got[60:], want[60:])
    K2.check_device_error()


def test_lora_fused_adapters_of_stacked_projections(K2):
    # separate adapters of four projections as one adapter of the stacked weight
    g = torch.Generator(device="cuda").manual_seed(5)
    sizes, K = (256, 128, 128, 256), 256
    parts = [[((torch.randn(r, K, device="cuda", generator=g) * K ** -0.5).bfloat16(),
               (torch.randn(n, r, device="cuda", generator=g) * 0.3).bfloat16()) for n, r in zip(sizes, rs)]
             for rs in ((8, 4, 4, 8), (3, 5, 8, 2))]
    lora = K2.LoraAdapters.fused(parts, torch.tensor([1.0, 0.5], device="cuda"))
    assert lora.rank == 24 and lora.Nw == sum(sizes)
    A = torch.randn(50, K, device="cuda", generator=g).bfloat16()
    W = (torch.randn(sum(sizes), K, device="cuda", generator=g) * K ** -0.5).bfloat16()
    start = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    ids = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    out = torch.empty(50, sum(sizes), device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(K2.lora_workspace_size(torch.bfloat16, K2.KREA2_EPI_STORE, 50, sum(sizes), K, 2, 24),
                     dtype=torch.uint8, device="cuda")
    K2.lora_linear(K2.KREA2_EPI_STORE, A, W, lora, start, ids, out, ws)
    K2.check_device_error()
    ref = A.double() @ W.double().T
    for (a, b), p, sc in (((0, 20), parts[1], 0.5), ((20, 50), parts[0], 1.0)):
        ref[a:b] += sc * torch.cat([(A[a:b].double() @ d.double().T) @ u.double().T for d, u in p], 1)
    rel, big = off(out, ref)
    assert rel <= TOL_BF16 and big <= 8 * TOL_BF16


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def one_tile_is_narrow(N):
    # gemm_bf16_lora's choice between 64 and 128 columns for one row tile
    def eff(tiles):
        return tiles / (-(-tiles // sms()) * sms())
    return eff(N // 64) > 1.25 * eff(N // 128)


@pytest.mark.parametrize("epilogue", ["store", "resid"])
@pytest.mark.parametrize("rows,spare,rank,K", [([1], 0, 16, 320), ([40, 0, 36, 1], 0, 64, 320), ([70, 7], 51, 24, 704),
                                               ([128], 0, 256, 448), ([1] * 128, 0, 8, 64)])
def test_lora_one_row_tile_in_128_columns(K2, epilogue, rows, spare, rank, K):
    # K of an odd number of 64-column steps: a stage holds two, the last one is filled up with zeros
    assert not one_tile_is_narrow(15360) and one_tile_is_narrow(768)
    Case(K2, epilogue, rows, K, 15360, rank, 3, torch.bfloat16, ids=[0, -1, 2, 1][:len(rows)] if len(rows) < 5 else None,
         spare=spare).check()


@pytest.mark.parametrize("epilogue,N", [("store", 2048), ("store", 2010), ("resid", 2048), ("resid", 1999),
                                        ("swiglu", 2048)])
@pytest.mark.parametrize("rank", [8, 40])
def test_lora_f32_large_tiles(K2, epilogue, N, rank):
    # 64 x 128 tiles are taken from two per SM on; rows, columns and K end inside tiles
    rows, K = [700, 0, 1, 599], 100
    assert -(-N // 128) * -(-(sum(rows) + 9) // 64) >= 2 * sms()
    Case(K2, epilogue, rows, K, N, rank, 3, torch.float32, ids=[2, 0, -1, 1], spare=9).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lora_overlapping_calls(K2, dtype):
    # two streams with calls in flight at once, each with its own workspace and outputs
    cases = [Case(K2, "store", [1, 70, 200], 1024, 1536, 48, 3, dtype, seed=1),
             Case(K2, "store", [33, 129], 512, 768, 16, 2, dtype, seed=2)]
    want = [c.run() for c in cases]
    turns = 20
    outs = [[torch.empty_like(c.out0) for _ in range(turns)] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(turns):
        for k in ((0, 1), (1, 0))[i % 2]:
            c = cases[k]
            K2.lora_linear(c.epi, c.A, c.W, c.lora, c.row_start, c.adapter, outs[k][i], c.ws, stream=streams[k])
    torch.cuda.synchronize()
    K2.check_device_error()
    for c, w, os in zip(cases, want, outs):
        for o in os:
            assert torch.equal(o[:c.used], w[:c.used])
