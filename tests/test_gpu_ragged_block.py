"""The ragged-batch operators together, as a server's step runs them: one transformer block over requests of different
lengths, each with its own adapter, modulation and cached keys, captured once and replayed with other lengths."""
import pytest
import torch

import krea2_inputs as KI
from ragged_ref import F64, Ragged, lora_ref, norm_rope, off

pytestmark = pytest.mark.gpu

BF16_RMS = 2.0 ** -8 / 3 ** 0.5
# Roundings to bf16 in series on the way into the residual: xn, the projection, the cached keys, q_hat, the
# probabilities, the attention's output; then xn2 and the activation, on inputs that the first branch moved.
TOL_BRANCH = 8 * BF16_RMS

D = KI.Dims(C=512, H=4, Hkv=1, D=128, F=768, axes=(32, 48, 48))
N_AD, RANK = 3, 16


@pytest.fixture(scope="module")
def K2(cuda_device):
    import flow_matching_stream_b200 as K2
    return K2


class Weights:
    def __init__(self, K2):
        g = torch.Generator(device="cuda").manual_seed(3)

        def rnd(*shape, scale=1.0, dt=torch.bfloat16):
            return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt)

        C, F, HD = D.C, D.F, D.HD
        self.lin, self.ad, self.lora = {}, {}, {}
        for name, (n, k) in {"qkvg": (D.qkvg_cols, C), "out": (C, HD), "gu": (2 * F, C), "down": (C, F)}.items():
            self.lin[name] = rnd(n, k, scale=k ** -0.5)
            self.ad[name] = (rnd(N_AD, RANK, k, scale=k ** -0.5), rnd(N_AD, n, RANK, scale=0.5 * RANK ** -0.5))
        self.scale = torch.rand(N_AD, device="cuda", generator=g) + 0.5
        for name, (down, up) in self.ad.items():
            self.lora[name] = K2.LoraAdapters(down, up, self.scale)
        f32 = torch.float32
        self.n1, self.n2, self.table = rnd(C, scale=0.1, dt=f32), rnd(C, scale=0.1, dt=f32), rnd(6, C, scale=0.1, dt=f32)


def rms(h, w, eps):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * (1 + w.to(F64))


class Step:
    """Buffers of up to `rows` new tokens of R requests, and the block's launches on them."""

    def __init__(self, K2, w, R, rows, pages, width, page):
        self.K2, self.w, self.R, self.rows = K2, w, R, rows
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, device="cuda", dtype=dt)  # noqa: E731
        i32, f32 = torch.int32, torch.float32
        self.q_start, self.kv_len, self.table = z(R + 1, dt=i32), z(R, dt=i32), z(R, width, dt=i32)
        self.adapter = z(R, dt=i32)
        self.kp, self.vp = z(pages, page, D.KVD), z(pages, page, D.KVD)
        self.h, self.temb, self.gates = z(rows, D.C, dt=f32), z(rows, 6 * D.C, dt=f32), z(2, R, D.C, dt=f32)
        self.cos, self.sin = z(rows, 64, dt=f32), z(rows, 64, dt=f32)
        self.qw, self.kw = z(128, dt=f32), z(128, dt=f32)
        self.xn, self.qkvg = z(rows, D.C), z(rows, D.qkvg_cols)
        self.attn, self.u = z(rows, D.HD), z(rows, D.F)
        self.batch = K2.PagedBatch(self.q_start, self.kv_len, self.table, self.kp, self.vp, rows)
        bf = torch.bfloat16
        need = max([K2.paged_attention_workspace_size(D, self.batch, bf)] +
                   [K2.lora_workspace_size(bf, 0, rows, *w.lin[n].shape, R, RANK) for n in w.lin])
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")  # one after the other on one stream

    def run(self):
        K2, w = self.K2, self.w

        def linear(epi, x, name, out, gate=None):
            K2.lora_linear(epi, x, w.lin[name], w.lora[name], self.q_start, self.adapter, out, self.ws, gate=gate)

        K2.modulated_rmsnorm(D, self.rows, 1, self.h, w.n1, self.temb, w.table, 0, self.xn)
        linear(K2.KREA2_EPI_STORE, self.xn, "qkvg", self.qkvg)
        K2.paged_kv_append(D, self.batch, self.qkvg, self.kw, self.cos, self.sin)
        K2.gqa_attention_paged(D, self.batch, self.qkvg, self.qw, self.cos, self.sin, None, None, self.attn, self.ws)
        linear(K2.KREA2_EPI_RESID, self.attn, "out", self.h, self.gates[0])
        K2.modulated_rmsnorm(D, self.rows, 1, self.h, w.n2, self.temb, w.table, 3, self.xn)
        linear(K2.KREA2_EPI_SWIGLU, self.xn, "gu", self.u)
        linear(K2.KREA2_EPI_RESID, self.u, "down", self.h, self.gates[1])


def reference(w, b, h0, temb, gates, ids):
    """The block in fp64 on the batch's rows; the cache's new keys and values are the block's own."""
    n, start = b.start[-1], b.start
    mod = temb[:n].to(F64).view(n, 6, D.C) + w.table.to(F64)
    h = h0[:n].to(F64)

    def linear(x, name, epi, out0=None, gate=None):
        rows_out = torch.zeros(n, w.lin[name].shape[0] // (2 if epi == "swiglu" else 1), dtype=F64, device="cuda")
        return lora_ref(x, w.lin[name], *w.ad[name], w.scale, start, ids, epi, rows_out if out0 is None else out0, gate)

    qkvg = linear((1 + mod[:, 0]) * rms(h, w.n1, D.eps) + mod[:, 1], "qkvg", "store")
    kp, vp = b.k_pages.to(F64), b.v_pages.to(F64)
    for r in range(b.R):
        if b.new[r] == 0:
            continue
        p, s = b.slots(r)
        sl, m = b.rowsof(r), b.new[r]
        k = norm_rope(qkvg[sl, D.HD:D.HD + D.KVD].reshape(m, D.Hkv, 128), b.kw, b.cos[sl], b.sin[sl], D.eps)
        kp[p[-m:], s[-m:]] = k.reshape(m, D.KVD)
        vp[p[-m:], s[-m:]] = qkvg[sl, D.HD + D.KVD:D.HD + 2 * D.KVD]
    b.qkvg = qkvg
    o, _ = b.attention(k_pages=kp, v_pages=vp)
    h = linear(o[:n], "out", "resid", h, gates[0])
    u = linear((1 + mod[:, 3]) * rms(h, w.n2, D.eps) + mod[:, 4], "gu", "swiglu")
    return linear(u, "down", "resid", h, gates[1])


def test_block_step_of_a_ragged_batch(K2):
    w = Weights(K2)
    cases = [([300, 1, 64, 0], [420, 777, 64, 30], [0, -1, 2, 1]), ([1, 1, 1, 1], [900, 65, 1, 300], [2, 2, -1, 0]),
             ([17, 200, 3, 90], [17, 500, 1030, 91], [1, 0, 1, 2])]
    bs = [Ragged(D, n, k, 16, torch.bfloat16, "cuda", seed=i) for i, (n, k, _) in enumerate(cases)]
    rows = 380
    st = Step(K2, w, 4, rows, max(b.num_pages for b in bs), max(b.max_pages for b in bs), 16)
    g = torch.Generator(device="cuda").manual_seed(9)
    st.q_start.copy_(bs[0].q_start), st.kv_len.copy_(bs[0].kv_len), st.table[:, :bs[0].max_pages].copy_(bs[0].table)
    st.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for b, (_, _, ids) in zip(bs, cases):
        n = b.rows
        st.q_start.copy_(b.q_start), st.kv_len.copy_(b.kv_len)
        st.table[:, :b.max_pages] = b.table
        st.kp[:b.num_pages], st.vp[:b.num_pages] = b.k_pages, b.v_pages
        st.cos[:n], st.sin[:n], st.qw[:], st.kw[:] = b.cos, b.sin, b.qw, b.kw
        st.adapter.copy_(torch.tensor(ids, dtype=torch.int32))
        st.h.copy_(torch.randn(rows, D.C, device="cuda", generator=g))
        st.temb.copy_(torch.randn(rows, 6 * D.C, device="cuda", generator=g) * 0.3)
        st.gates.copy_(torch.randn(2, 4, D.C, device="cuda", generator=g) * 0.5)
        h0 = st.h.clone()
        ref = reference(w, b, h0, st.temb, st.gates, ids)
        graph.replay()
        K2.check_device_error()
        rel, _ = off(st.h[:n] - h0[:n], ref - h0[:n].to(F64))
        assert rel <= TOL_BRANCH
        assert torch.equal(st.h[n:], h0[n:])  # rows behind the last request
