"""Serving operators of a ragged batch of requests: attention of new tokens over a paged key/value
cache, the append that fills its pages, and a projection with low-rank adapters per request.

Each case is a dict of plain values. `prepare` draws its inputs on the GPU from a seed, `run` makes one
pass: with `own` false in elementary torch operations in fp32, with `own` true through
flow_matching_stream_b200. `exact` gives the same outputs in fp64, written apart from both.
"""
import itertools
import math
import random

import numpy as np
import torch

own = False

# Krea2Transformer2DModel's default block, and the tiny test configuration of this repository.
FULL = {"C": 6144, "H": 48, "Hkv": 12, "D": 128, "F": 16384, "axes": (32, 48, 48), "theta": 1000.0, "eps": 1e-5}
TINY = {"C": 256, "H": 4, "Hkv": 1, "D": 64, "F": 512, "axes": (16, 24, 24), "theta": 1000.0, "eps": 1e-5}
MODELS = {"full": FULL, "tiny": TINY}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class Dims:
    """The hyper-parameters that an entry point's `dims` argument reads."""

    def __init__(self, m):
        for k, v in m.items():
            setattr(self, k, v)
        self.n_layers, self.in_ch, self.t_dim = 1, 64, 256


class State:
    pass


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one text token of one short conversation: the smallest call, where latency counts
        {"name": "attn_1tok_short", "op": "attention", "model": "full", "dtype": "bf16", "new": "1", "kv": "77",
         "page": 16, "T": 0, "causal": False, "spare": 0},
        # eight requests, one new token each, behind cached prompts and condition images of several sizes
        {"name": "attn_1tok_8req", "op": "attention", "model": "full", "dtype": "bf16", "new": "1,1,1,1,1,1,1,1",
         "kv": "521,1537,8704,4609,2817,4608,8191,6400", "page": 64, "T": 512, "causal": False, "spare": 0},
        # two 1024^2 images being denoised after a cached prompt and condition image of the same size
        {"name": "attn_denoise_2req", "op": "attention", "model": "full", "dtype": "bf16", "new": "4096,4096",
         "kv": "8704,8703", "page": 64, "T": 512, "causal": False, "spare": 0},
        # a mixed batch: prompts being read causally in chunks beside requests that take one token each
        {"name": "attn_mixed_causal", "op": "attention", "model": "full", "dtype": "bf16",
         "new": "1,301,37,1229,1,512,128", "kv": "4097,301,1061,5325,77,1536,2175", "page": 16, "T": 0, "causal": True,
         "spare": 19},
        # the tiny fp32 configuration, for reference precision
        {"name": "attn_tiny_f32", "op": "attention", "model": "tiny", "dtype": "f32", "new": "64,8,1",
         "kv": "72,75,130", "page": 16, "T": 8, "causal": False, "spare": 0},
        # the keys and values of one new token of each of eight requests
        {"name": "append_1tok_8req", "op": "append", "model": "full", "dtype": "bf16", "new": "1,1,1,1,1,1,1,1",
         "kv": "521,1537,8704,4609,2817,4608,8191,6400", "page": 64, "spare": 0},
        # two 1024^2 images' keys and values behind a cached prompt and condition image
        {"name": "append_denoise_2req", "op": "append", "model": "full", "dtype": "bf16", "new": "4096,4096",
         "kv": "8704,8703", "page": 64, "spare": 0},
        # to_out of one new token with its request's adapter: the weight's bytes and latency
        {"name": "lora_out_1row", "op": "lora", "dtype": "bf16", "epilogue": "store", "K": 6144, "N": 6144, "rank": 16,
         "rows": "1", "adapters": 4, "spare": 0},
        # the fused projection of a ragged batch: prompts, single tokens and a 512^2 image, one without an adapter
        {"name": "lora_qkvg_mixed", "op": "lora", "dtype": "bf16", "epilogue": "store", "K": 6144, "N": 15360,
         "rank": 64, "rows": "1,301,37,1024,1,128,77,1", "adapters": 6, "spare": 19},
        # gate/up with SwiGLU of one 1024^2 image with its prompt, and of a second, smaller one
        {"name": "lora_gate_up", "op": "lora", "dtype": "bf16", "epilogue": "swiglu", "K": 6144, "N": 32768, "rank": 16,
         "rows": "4608,1152", "adapters": 2, "spare": 0},
        # down with the gated residual of four requests with prompts of different lengths
        {"name": "lora_down_resid", "op": "lora", "dtype": "bf16", "epilogue": "resid", "K": 16384, "N": 6144,
         "rank": 32, "rows": "1152,1101,1029,1536", "adapters": 4, "spare": 0},
        # the tiny fp32 configuration's fused projection
        {"name": "lora_tiny_f32", "op": "lora", "dtype": "f32", "epilogue": "store", "K": 256, "N": 640, "rank": 8,
         "rows": "64,8,1", "adapters": 2, "spare": 0},
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "lora", "lora"])
    small = rng.random() < 0.15
    R = log_int(rng, 1, 12)
    spare = rng.choice([0, 0, rng.randint(1, 200)])
    if op == "lora":
        rows = [log_int(rng, 1, 3500 if i == 0 else 200) for i in range(R)]
        rng.shuffle(rows)
        m = TINY if small else FULL
        QC = 2 * m["H"] * m["D"] + 2 * m["Hkv"] * m["D"]
        K, N, epi = rng.choice([(m["C"], QC, "store"), (m["C"], m["C"], "store"), (m["C"], m["C"], "resid"),
                                (m["C"], 2 * m["F"], "swiglu"), (m["F"], m["C"], "resid")])
        if small:
            rows = [1 + r // 32 for r in rows]
        return {"op": op, "dtype": "f32" if small else "bf16", "epilogue": epi, "K": K, "N": N,
                "rank": 8 * log_int(rng, 1, 16), "rows": text(rows), "adapters": rng.randint(1, R + 1),
                "spare": spare}
    top = 130 if small else 12000
    new, kv = [], []
    for i in range(R):
        n = 1 if rng.random() < 0.4 else log_int(rng, 1, 64 if small else (4096 if i == 0 else 600))
        new.append(n)
        kv.append(max(n, log_int(rng, 16, top)))
    most = max(1, 2 * 4096 * 8704 // (R * max(kv)))  # the largest listed case, with every request padded to the longest
    new = [min(n, most) for n in new]
    c = {"op": op, "model": "tiny" if small else "full", "dtype": "f32" if small else "bf16", "new": text(new),
         "kv": text(kv), "page": rng.choice([16, 32, 64, 128]), "spare": spare}
    if op == "attention":
        c["T"] = rng.choice([0, 8, 77, 512])
        c["causal"] = rng.random() < 0.5
    return c


def ints(s):
    return [int(v) for v in s.split(",")]


# ------------------------------------------------------------------------------------------ inputs

def normal(g, shape, std, dtype):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def rope_tables(m, positions):
    """cos, sin (rows, D/2) of (t, h, w) positions, angles in fp64."""
    angle = torch.cat([positions[:, a, None] * m["theta"] ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
                       for a, d in enumerate(m["axes"])], 1)
    return torch.cos(angle).float().contiguous(), torch.sin(angle).float().contiguous()


def make_paged(case, seed):
    """The batch of a paged case: new tokens' raw projection, lengths, pages in random order, RoPE tables."""
    s = State()
    m = s.m = MODELS[case["model"]]
    dt = DTYPES[case["dtype"]]
    new, kv, page = ints(case["new"]), ints(case["kv"]), case["page"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    R, rows = len(new), sum(new) + case["spare"]
    start = list(itertools.accumulate(new, initial=0))
    per = [-(-n // page) for n in kv]
    max_pages = max(per) + 1
    order = list(range(sum(per) + 3))
    rng.shuffle(order)
    table = [[order.pop() if i < per[r] else -1 for i in range(max_pages)] for r in range(R)]
    s.new, s.kv, s.R, s.rows, s.page, s.start = new, kv, R, rows, page, start
    s.q_start, s.kv_len, s.page_table = i32(start), i32(kv), i32(table)
    HD, KVD = m["H"] * m["D"], m["Hkv"] * m["D"]
    s.qkvg = normal(g, (rows, 2 * HD + 2 * KVD), 1.0, dt)
    pool = (sum(per) + 3, page, KVD)
    s.k_pages, s.v_pages = normal(g, pool, 1.0, dt), normal(g, pool, 1.0, dt)
    s.q_norm_w, s.k_norm_w = normal(g, (m["D"],), 0.1, torch.float32), normal(g, (m["D"],), 0.1, torch.float32)
    at = np.concatenate([np.arange(kv[r] - new[r], kv[r]) for r in range(R)] + [np.zeros(case["spare"])])
    s.cos, s.sin = rope_tables(m, torch.from_numpy(np.stack([0 * at, at // 64, at % 64], 1)).cuda())
    s.text_mask = s.key_end = None
    if case["op"] == "attention":
        s.T = T = min(case["T"], min(kv))
        if T:
            keep = [rng.randint(1, T) for _ in range(R)]  # right-padded prompts
            s.text_mask = i32([[int(i < keep[r]) for i in range(T)] for r in range(R)]).to(torch.uint8)
        if case["causal"]:
            s.key_end = i32([kv[r] - new[r] + i + 1 for r in range(R) for i in range(new[r])] + [0] * case["spare"])
        s.out = torch.zeros(rows, HD, device="cuda", dtype=dt)
    return s


def make_lora(case, seed):
    s = State()
    dt = DTYPES[case["dtype"]]
    rows, K, N, rank, n_ad = ints(case["rows"]), case["K"], case["N"], case["rank"], case["adapters"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    R, M = len(rows), sum(rows) + case["spare"]
    start = list(itertools.accumulate(rows, initial=0))
    s.R, s.M, s.start, s.epilogue = R, M, start, case["epilogue"]
    s.ids = [rng.randrange(n_ad) for _ in range(R)]
    if R > 2:
        s.ids[R // 2] = -1  # a request without an adapter
    s.row_start, s.adapter = i32(start), i32(s.ids)
    s.A = normal(g, (M, K), 1.0, dt)
    s.W = normal(g, (N, K), K ** -0.5, dt)
    s.down = normal(g, (n_ad, rank, K), K ** -0.5, dt)
    s.up = normal(g, (n_ad, N, rank), 0.5 * rank ** -0.5, dt)
    s.scale = torch.rand(n_ad, device="cuda", generator=g) + 0.5
    if s.epilogue == "resid":
        s.gate = normal(g, (R, N), 0.5, torch.float32)
        s.out = normal(g, (M, N), 1.0, torch.float32)
    else:
        s.gate = None
        s.out = torch.zeros(M, N // 2 if s.epilogue == "swiglu" else N, device="cuda", dtype=dt)
    return s


def prepare(case, seed):
    s = make_lora(case, seed) if case["op"] == "lora" else make_paged(case, seed)
    s.op, s.dtype = case["op"], DTYPES[case["dtype"]]
    if own:
        import flow_matching_stream_b200 as K2
        s.K2 = K2
        if s.op == "lora":
            s.epi = {"store": K2.KREA2_EPI_STORE, "swiglu": K2.KREA2_EPI_SWIGLU, "resid": K2.KREA2_EPI_RESID}[s.epilogue]
            s.lora = K2.LoraAdapters(s.down, s.up, s.scale)
            n = K2.lora_workspace_size(s.dtype, s.epi, s.M, s.W.shape[0], s.W.shape[1], s.R, s.lora.rank)
        else:
            s.dims = K2.dims_struct(Dims(s.m))
            s.batch = K2.PagedBatch(s.q_start, s.kv_len, s.page_table, s.k_pages, s.v_pages, s.rows)
            n = K2.paged_attention_workspace_size(s.dims, s.batch, s.dtype) if s.op == "attention" else 0
        s.ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------------------- one pass

def norm_rope(x, w, cos, sin, eps):
    """(rows, heads, D) fp32: RMSNorm with (1 + w), then rotation of adjacent pairs by the row's angles."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (1 + w)
    a, b = x[..., 0::2], x[..., 1::2]
    c, s = cos[:, None], sin[:, None]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


def row_requests(start, rows):
    """Request of each of the first `rows` rows, and the row's index in it."""
    at = torch.arange(rows, device="cuda")
    req = torch.searchsorted(start, at, right=True) - 1
    return req, at - start[req]


def plain_attention(s):
    m, H, Hkv, D = s.m, s.m["H"], s.m["Hkv"], s.m["D"]
    HD, KVD, R, G = H * D, Hkv * D, s.R, H // Hkv
    used, N, L = s.start[-1], max(s.new), max(s.kv)
    start, kv_len = s.q_start.long(), s.kv_len.long()
    x = s.qkvg[:used].float()
    q = norm_rope(x[:, :HD].view(used, H, D), s.q_norm_w, s.cos[:used], s.sin[:used], m["eps"])
    gate = torch.sigmoid(x[:, HD + 2 * KVD:])
    at = torch.arange(N, device="cuda")
    rows = (start[:-1, None] + at).clamp(max=used - 1)  # (R, N), padded by rows that are dropped below
    pages = s.page_table[:, :-(-L // s.page)].long().clamp(min=0)
    k = s.k_pages[pages].reshape(R, -1, Hkv, D)[:, :L].float().permute(0, 2, 3, 1)
    v = s.v_pages[pages].reshape(R, -1, Hkv, D)[:, :L].float().permute(0, 2, 1, 3)
    qp = q[rows].view(R, N, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * N, D)
    key = torch.arange(L, device="cuda")
    seen = (key < kv_len[:, None])[:, None].expand(R, N, L)
    if s.key_end is not None:
        own_end = (kv_len - start.diff())[:, None] + at + 1
        seen = seen & (key < torch.maximum(s.key_end.long()[rows], own_end)[..., None])
    if s.text_mask is not None:
        padded = torch.cat([s.text_mask == 0, torch.zeros(R, L - s.T, dtype=torch.bool, device="cuda")], 1)
        seen = seen & ~padded[:, None]
    scores = (qp @ k).mul_(D ** -0.5).view(R, Hkv, G, N, L)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(R, Hkv, G * N, L) @ v).view(R, Hkv, G, N, D) / torch.where(total == 0, torch.ones_like(total), total)
    req, i = row_requests(start, used)
    o = o.permute(0, 3, 1, 2, 4).reshape(R, N, HD)[req, i] * gate
    out = torch.zeros(s.rows, HD, device="cuda", dtype=s.dtype)
    out[:used] = o.to(s.dtype)
    return out


def plain_append(s):
    m, H, Hkv, D = s.m, s.m["H"], s.m["Hkv"], s.m["D"]
    HD, KVD, used = H * D, Hkv * D, s.start[-1]
    start = s.q_start.long()
    k = norm_rope(s.qkvg[:used, HD:HD + KVD].float().view(used, Hkv, D), s.k_norm_w, s.cos[:used], s.sin[:used],
                  m["eps"])
    req, i = row_requests(start, used)
    pos = (s.kv_len.long() - start.diff())[req] + i
    page = s.page_table.long()[req, pos // s.page]
    s.k_pages[page, pos % s.page] = k.reshape(used, KVD).to(s.dtype)
    s.v_pages[page, pos % s.page] = s.qkvg[:used, HD + KVD:HD + 2 * KVD]
    return s.k_pages, s.v_pages


def plain_lora(s):
    used = s.start[-1]
    x = s.A[:used].float()
    y = x @ s.W.float().t()
    n_ad, rank, K = s.down.shape
    req, _ = row_requests(s.row_start.long(), used)
    ids = s.adapter.long()[req]
    pick = (ids[:, None] == torch.arange(n_ad, device="cuda")).float() * s.scale  # rows without an adapter: zeros
    t = (x @ s.down.float().view(n_ad * rank, K).t()).view(used, n_ad, rank) * pick[..., None]
    y += t.view(used, n_ad * rank) @ s.up.float().transpose(1, 2).reshape(n_ad * rank, -1)
    if s.epilogue == "resid":
        s.out[:used] += s.gate[req] * y
        return s.out
    if s.epilogue == "swiglu":  # W's rows alternate 64 of the gate and 64 of the up projection
        y = y.view(used, -1, 2, 64)
        y = (y[:, :, 0] * torch.sigmoid(y[:, :, 0]) * y[:, :, 1]).reshape(used, -1)
    out = torch.zeros_like(s.out)
    out[:used] = y.to(s.dtype)
    return out


def run(s):
    if own:
        K2 = s.K2
        if s.op == "attention":
            K2.gqa_attention_paged(s.dims, s.batch, s.qkvg, s.q_norm_w, s.cos, s.sin, s.text_mask, s.key_end, s.out,
                                   s.ws)
            return s.out
        if s.op == "append":
            K2.paged_kv_append(s.dims, s.batch, s.qkvg, s.k_norm_w, s.cos, s.sin)
            return s.k_pages, s.v_pages
        K2.lora_linear(s.epi, s.A, s.W, s.lora, s.row_start, s.adapter, s.out, s.ws, gate=s.gate)
        return s.out
    return {"attention": plain_attention, "append": plain_append, "lora": plain_lora}[s.op](s)


# ------------------------------------------------------------------------------------- what it costs

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "lora":
        rows, K, N, rank = ints(case["rows"]), case["K"], case["N"], case["rank"]
        M = sum(rows)
        adapted = len(rows) - (1 if len(rows) > 2 else 0)
        used = min(case["adapters"], adapted)
        out = {"store": M * N * es, "swiglu": M * N // 2 * es, "resid": 2 * M * N * 4 + len(rows) * N * 4}
        return {"bytes": (M * K + N * K + used * rank * (K + N)) * es + out[case["epilogue"]],
                "flops": 2.0 * M * N * K + 2.0 * M * rank * (K + N) * adapted / len(rows)}
    m = MODELS[case["model"]]
    H, Hkv, D = m["H"], m["Hkv"], m["D"]
    new, kv = ints(case["new"]), ints(case["kv"])
    M, tables = sum(new), sum(new) * D * 4
    if case["op"] == "append":
        return {"bytes": 4.0 * M * Hkv * D * es + tables, "flops": 10.0 * M * Hkv * D}
    seen = 0
    for n, L in zip(new, kv):
        seen += n * L - (n * (n - 1) // 2 if case["causal"] else 0)
    return {"bytes": (3.0 * M * H * D + 2.0 * sum(kv) * Hkv * D) * es + tables, "flops": 4.0 * seen * H * D}


# ----------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["op"] == "lora":
        s = make_lora(case, seed)
        out = s.out.double()
        for r in range(s.R):
            a, b = s.start[r], s.start[r + 1]
            for c in range(a, b, 1024):
                x = s.A[c:min(b, c + 1024)].double()
                y = torch.mm(x, s.W.double().T)
                j = s.ids[r]
                if j >= 0:
                    y += s.scale[j].double() * torch.mm(torch.mm(x, s.down[j].double().T), s.up[j].double().T)
                if s.epilogue == "resid":
                    y = out[c:c + len(x)] + s.gate[r].double() * y
                elif s.epilogue == "swiglu":
                    y = torch.cat([y[:, n:n + 64] / (1 + torch.exp(-y[:, n:n + 64])) * y[:, n + 64:n + 128]
                                   for n in range(0, y.shape[1], 128)], 1)
                out[c:c + len(x)] = y
        return out
    s = make_paged(case, seed)
    m = s.m
    H, Hkv, D = m["H"], m["Hkv"], m["D"]

    def head(row0, row1, first, h, w):  # one head of the rows' raw projection, normalised and turned as complex pairs
        y = s.qkvg[row0:row1, first + h * D:first + (h + 1) * D].double()
        y = y / torch.sqrt(y.square().sum(1, keepdim=True) / D + m["eps"]) * (1 + w.double())
        z = torch.view_as_complex(y.view(row1 - row0, D // 2, 2).contiguous())
        turn = torch.complex(s.cos[row0:row1].double(), s.sin[row0:row1].double())
        return torch.view_as_real(z * turn).reshape(row1 - row0, D)

    if case["op"] == "append":
        k, v = s.k_pages.double(), s.v_pages.double()
        for r in range(s.R):
            n, a, b = s.new[r], s.start[r], s.start[r + 1]
            pos = torch.arange(s.kv[r] - n, s.kv[r], device="cuda")
            page, slot = s.page_table[r].long()[torch.div(pos, s.page, rounding_mode="floor")], pos % s.page
            for h in range(Hkv):
                k[page, slot, h * D:(h + 1) * D] = head(a, b, H * D, h, s.k_norm_w)
            v[page, slot] = s.qkvg[a:b, (H + Hkv) * D:(H + 2 * Hkv) * D].double()
        return k, v
    out = torch.zeros(s.rows, H * D, dtype=torch.float64, device="cuda")
    for r in range(s.R):
        n, L, a, b = s.new[r], s.kv[r], s.start[r], s.start[r + 1]
        pages = s.page_table[r, :-(-L // s.page)].long()
        hidden = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if s.text_mask is not None:
            hidden[:, :s.T] |= s.text_mask[r] == 0
        if s.key_end is not None:
            ends = torch.maximum(s.key_end[a:b].long(), torch.arange(L - n + 1, L + 1, device="cuda"))
            hidden |= torch.arange(L, device="cuda")[None] >= ends[:, None]
        for h in range(H):
            j = h // (H // Hkv) * D
            k = s.k_pages[pages, :, j:j + D].reshape(-1, D)[:L].double()
            v = s.v_pages[pages, :, j:j + D].reshape(-1, D)[:L].double()
            z = torch.mm(head(a, b, 0, h, s.q_norm_w), k.T) / math.sqrt(D)
            p = torch.nan_to_num(torch.softmax(z.masked_fill(hidden, -math.inf), 1), nan=0.0)
            g = s.qkvg[a:b, (H + 2 * Hkv + h) * D:(H + 2 * Hkv + h + 1) * D].double()
            out[a:b, h * D:(h + 1) * D] = torch.mm(p, v) / (1 + torch.exp(-g))
    return out
