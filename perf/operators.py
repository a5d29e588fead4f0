"""The latent-cache operators, as they are measured: inputs, plain forms, calls and exact results.

Operators (576 cached values a token: a 512-value latent and a 64-value shared rope key):
  latent     Indexer.latent_attention: absorbed form, every query attends to its whole causal
             prefix (prompt chunks, drafted tokens, single decode tokens)
  fp4        Indexer.latent_attention_fp4: the same over a cache held in 4 bits
  fp4sel     Indexer.latent_attention_fp4 over the positions an index row selects
  quant      Indexer.quantize_latent_fp4 and dequantize_latent_fp4: rows into that cache and back
  expanded   Indexer.latent_attention_expanded: per-head keys and values up-projected from the
             latent, for prompts
"""

import math
import random

import torch

own = False

LATENT, ROPE, DIM = 512, 64, 576
NOPE, HEAD_QK, HEAD_V = 128, 192, 128
SCALE = HEAD_QK ** -0.5
ROW4 = LATENT // 2 + LATENT // 16 + 2 * ROPE      # bytes of a 4-bit row: codes, block scales, rope key
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # magnitudes of the 4-bit codes


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a chat that has just begun: nothing but latency
        dict(name="latent_one_short", op="latent", batch=1, l_min=37, l_max=37, nq=1, heads=96, lens_seed=1),
        # the decode batch of the benchmark: 64 sequences of 16,384..131,072 tokens, one query each
        dict(name="latent_decode_64", op="latent", batch=64, l_min=16384, l_max=131072, nq=1, heads=96, lens_seed=2),
        # three drafted tokens a sequence, half the heads on this GPU, ragged lengths
        dict(name="latent_draft_8", op="latent", batch=8, l_min=2001, l_max=9001, nq=3, heads=48, lens_seed=3),
        # a chunk of a prompt appended to a cached prefix
        dict(name="latent_chunk_512", op="latent", batch=1, l_min=6145, l_max=6145, nq=512, heads=96, lens_seed=4),
        # a long-context decode batch whose cache is held in 4 bits
        dict(name="fp4_decode_32", op="fp4", batch=32, l_min=16384, l_max=65536, nq=1, heads=96, lens_seed=5),
        # few heads a GPU, short and ragged sequences
        dict(name="fp4_short_2", op="fp4", batch=2, l_min=1, l_max=200, nq=1, heads=16, lens_seed=6),
        # decode over the indexer's 2,048 selected positions, cache in 4 bits
        dict(name="fp4_selected_64", op="fp4sel", batch=64, l_min=8192, l_max=32768, nq=1, heads=96, k_sel=2048,
             lens_seed=7),
        # the rows of a prompt written into the 4-bit cache
        dict(name="quant_prompt_8k", op="quant", n=8191, scatter=False),
        # the new tokens of a decode batch, each to its own sequence's row
        dict(name="quant_decode_64", op="quant", n=64, scatter=True),
        # the 8,192-token prompt of the benchmark
        dict(name="expanded_8k", op="expanded", batch=1, l_min=8192, l_max=8192, nq=8192, heads=96, lens_seed=8),
        # a ragged batch of short prompts
        dict(name="expanded_ragged_5", op="expanded", batch=5, l_min=1, l_max=1501, nq=1501, heads=32, lens_seed=9),
        # a chunk of a long prompt, few heads a GPU
        dict(name="expanded_chunk_1k", op="expanded", batch=1, l_min=16001, l_max=16001, nq=1000, heads=16, lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("latent", "latent", "fp4", "fp4sel", "quant", "expanded", "expanded"))
    if op == "quant":
        return dict(op=op, n=_log_int(rng, 1, 30000), scatter=rng.random() < 0.5)
    heads = rng.choice((1, 6, 12, 16, 24, 32, 48, 64, 96))
    c = dict(op=op, heads=heads, lens_seed=rng.randrange(1, 1 << 30))
    if op == "expanded":
        c["batch"] = _log_int(rng, 1, 8)
        top = _log_int(rng, 1, 12000 // c["batch"])
        c["l_max"] = top
        c["l_min"] = rng.choice((1, max(1, top // 2), top))
        c["nq"] = rng.choice((top, top, max(1, top // 3)))
        while work(c)["flops"] > 2.0e12:
            c["heads"] = max(1, c["heads"] // 2)
    else:
        c["batch"] = _log_int(rng, 1, 96)
        top = _log_int(rng, 1, min(131072, 1500000 // c["batch"]))
        c["l_max"] = top
        c["l_min"] = rng.choice((1, max(1, top // 4), top))
        c["nq"] = rng.choice((1, 1, 1, 2, 4, _log_int(rng, 1, 300)))
        if op == "fp4sel":
            c["nq"] = min(c["nq"], 4)
            c["k_sel"] = rng.choice((2048, _log_int(rng, 1, 2048)))
        while work(c)["flops"] > 6.0e11:
            c["nq"] = max(1, c["nq"] // 2)
            c["batch"] = max(1, c["batch"] * 2 // 3)
    return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["l_min"], case["l_max"]) for _ in range(case["batch"])]
    return lens, [min(case["nq"], n) for n in lens]


def work(case):
    if case["op"] == "quant":
        n = case["n"]   # rows written, then read back
        return {"bytes": 2 * n * (2 * DIM + ROW4) + (16 * n if case["scatter"] else 0), "flops": 4 * n * LATENT}
    lens, nq = _lens(case)
    H, T = case["heads"], sum(nq)
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for n, q in zip(lens, nq))
    if case["op"] == "expanded":
        rows = sum(lens)
        return {"bytes": T * H * (2 * HEAD_QK + 2 * HEAD_V) + rows * 2 * DIM + H * 256 * LATENT * 2,
                "flops": pairs * H * 2 * (HEAD_QK + HEAD_V) + rows * H * 2 * 256 * LATENT}
    row = 2 * DIM if case["op"] == "latent" else ROW4
    rows = sum(lens)
    extra = 0
    if case["op"] == "fp4sel":
        # a query's selection holds min(k_sel, positions it may see) tokens
        sel = [min(case["k_sel"], n - q + j + 1) for n, q in zip(lens, nq) for j in range(q)]
        pairs = sum(sel)
        rows = min(rows, pairs)
        extra = T * case["k_sel"] * 4
    return {"bytes": rows * row + T * H * (2 * DIM + 2 * LATENT + 4) + extra,
            "flops": pairs * H * 2 * (DIM + LATENT)}


# ---------------------------------------------------------------------------------------- 4-bit rows

def _fp4_parts(x):
    """Block scales (fp32 values of e4m3) and code indices (sign in bit 3) of the latent part of x [n, 576]."""
    v = x[:, :LATENT].float().view(-1, LATENT // 16, 16)
    amax = v.abs().amax(-1)
    s = (amax.double() / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn).float()
    # nearest magnitude, ties to the even code: the exact products of a 3-bit midpoint and a 4-bit scale
    a = v.abs().double()
    mids = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    code = torch.zeros(v.shape, dtype=torch.uint8, device=x.device)
    for i, m in enumerate(mids):
        edge = (s.double() * m)[..., None]
        code += ((a > edge) if i % 2 == 0 else (a >= edge)).to(torch.uint8)
    code = torch.where((s > 0)[..., None], code, torch.zeros_like(code))
    code |= (torch.signbit(v) & (s > 0)[..., None]).to(torch.uint8) << 3
    return s, code


def _fp4_values(s, code):
    grid = torch.tensor(GRID, dtype=torch.float32, device=code.device)
    v = grid[(code & 7).long()] * s[..., None]
    return torch.where((code & 8) != 0, -v, v).reshape(code.shape[0], LATENT)


def _fp4_pack(x, out):
    """Rows of x as the 4-bit cache stores them (low nibble first)."""
    for i in range(0, x.shape[0], 1 << 18):
        y = x[i:i + (1 << 18)]
        s, code = _fp4_parts(y)
        code = code.reshape(y.shape[0], LATENT)
        out[i:i + (1 << 18), :256] = code[:, 0::2] | (code[:, 1::2] << 4)
        out[i:i + (1 << 18), 256:288] = s.to(torch.float8_e4m3fn).view(torch.uint8)
        out[i:i + (1 << 18), 288:] = y[:, LATENT:].contiguous().view(torch.uint8)


def _fp4_unpack(rows):
    """fp32 [n, 576] values of 4-bit rows."""
    b = rows[:, :256]
    code = torch.stack((b & 15, b >> 4), dim=-1).reshape(rows.shape[0], LATENT // 16, 16)
    s = rows[:, 256:288].contiguous().view(torch.float8_e4m3fn).float()
    rope = rows[:, 288:].contiguous().view(torch.bfloat16).float()
    return torch.cat((_fp4_values(s, code), rope), dim=1)


# ---------------------------------------------------------------------------------------- inputs

_INDEXER = []


def _indexer():
    """The layer's handle: a program makes it once."""
    if not _INDEXER:
        import dsa_lightning_indexer_03_b200 as dsa
        g = torch.Generator().manual_seed(0)
        w = [torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in ((64, 4096), (128, 128), (128, 32), (128,), (128,))]
        _INDEXER.append(dsa.Indexer(*w, max_tokens=4096))
    return _INDEXER[0]


def _randn(g, *shape):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda")
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    st = dict(case=case, ix=_indexer() if own else None)
    if case["op"] == "quant":
        n = case["n"]
        x = _randn(g, n, DIM)
        # a few channels run an order of magnitude larger, as latents' do; one block is empty
        x[:, torch.randperm(LATENT, generator=g, device="cuda")[:8]] *= 12
        x[n // 2, 32:48] = 0
        rows = torch.randperm(4 * n, generator=g, device="cuda")[:n] if case["scatter"] else None
        st.update(x=x, rows=rows, cache=torch.zeros((4 * n if case["scatter"] else n, ROW4), dtype=torch.uint8, device="cuda"))
        return st
    lens, nq = _lens(case)
    B, T, H, rows = len(lens), sum(nq), case["heads"], sum(lens)
    off = lambda v, t: torch.tensor([sum(v[:i]) for i in range(len(v) + 1)], dtype=t, device="cuda")  # noqa: E731
    st["lens"], st["nq"] = lens, nq
    st["q_off"], st["c_off"] = off(nq, torch.int32), off(lens, torch.int64)
    st["pos"] = torch.cat([torch.arange(n - q, n, dtype=torch.int32) for n, q in zip(lens, nq)]).cuda()
    st["q"] = _randn(g, T, H, HEAD_QK if case["op"] == "expanded" else DIM)
    kv = _randn(g, rows, DIM)
    if case["op"] in ("latent", "expanded"):
        st["kv"] = kv
    else:
        st["kv4"] = torch.empty((rows, ROW4), dtype=torch.uint8, device="cuda")
        _fp4_pack(kv, st["kv4"])
    if case["op"] == "expanded":
        # [H, 128 key rows then 128 value rows, 512], each row N(0, 1/512)
        st["w_ukv"] = _randn(g, H, 256, LATENT).mul_(LATENT ** -0.5)
    if case["op"] == "fp4sel":
        k = case["k_sel"]
        idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        for t, p in enumerate(st["pos"].tolist()):
            n = min(k, p + 1)
            idx[t, :n] = torch.randperm(p + 1, generator=g, device="cuda")[:n].to(torch.int32)
        st["idx"] = idx
    return st


# ---------------------------------------------------------------------------------------- one pass

def run(state):
    op, ix = state["case"]["op"], state["ix"]
    if own:
        if op == "quant":
            cache = ix.quantize_latent_fp4(state["x"], out=state["cache"], rows=state["rows"])
            return ix.dequantize_latent_fp4(cache, rows=state["rows"])
        a = (state["pos"], state["q_off"], state["c_off"], SCALE)
        if op == "latent":
            return ix.latent_attention(state["q"], state["kv"], *a)
        if op == "expanded":
            return ix.latent_attention_expanded(state["q"], state["kv"], state["w_ukv"], *a)
        return ix.latent_attention_fp4(state["q"], state["kv4"], *a, idx=state.get("idx"))
    if op == "quant":
        x = state["x"]
        return torch.cat((_fp4_values(*_fp4_parts(x)).to(torch.bfloat16), x[:, LATENT:]), dim=1)
    return _plain_expanded(state) if op == "expanded" else _plain_absorbed(state)


def _softmax_sums(s):
    """Weights and natural log of their sum along the last axis; every row has a finite score."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    return e / z, (m + torch.log(z)).squeeze(-1)


def _plain_absorbed(st):
    T, H = st["q"].shape[:2]
    out = torch.empty((T, H, LATENT), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, H), dtype=torch.float32, device="cuda")
    t0 = r0 = 0
    for n, nq in zip(st["lens"], st["nq"]):
        if "idx" in st:
            for t in range(t0, t0 + nq):
                sel = st["idx"][t]
                sel = sel[:min(sel.numel(), n - nq + t - t0 + 1)].long()
                c = _fp4_unpack(st["kv4"][r0 + sel])
                p, lse[t] = _softmax_sums(st["q"][t].float() @ c.t() * SCALE)
                out[t] = (p @ c[:, :LATENT]).to(torch.bfloat16)
        else:
            c = st["kv"][r0:r0 + n].float() if "kv" in st else _fp4_unpack(st["kv4"][r0:r0 + n])
            step = max(1, (1 << 28) // (n * H))
            for t in range(t0, t0 + nq, step):
                e = min(t + step, t0 + nq)
                s = st["q"][t:e].float() @ c.t() * SCALE                         # [queries, H, n]
                late = torch.arange(n, device="cuda") > st["pos"][t:e, None]
                p, lse[t:e] = _softmax_sums(s.masked_fill(late[:, None], -math.inf))
                out[t:e] = (p @ c[:, :LATENT]).to(torch.bfloat16)
        t0 += nq
        r0 += n
    return out, lse


def _plain_expanded(st):
    T, H = st["q"].shape[:2]
    out = torch.empty((T, H, HEAD_V), dtype=torch.bfloat16, device="cuda")
    t0 = r0 = 0
    for n, nq in zip(st["lens"], st["nq"]):
        c = st["kv"][r0:r0 + n].float()
        late = torch.arange(n, device="cuda") > st["pos"][t0:t0 + nq, None]
        for h in range(H):
            kv = c[:, :LATENT] @ st["w_ukv"][h].float().t()
            k = torch.cat((kv[:, :NOPE], c[:, LATENT:]), dim=1)
            s = st["q"][t0:t0 + nq, h].float() @ k.t() * SCALE
            p, _ = _softmax_sums(s.masked_fill_(late, -math.inf))
            out[t0:t0 + nq, h] = (p @ kv[:, NOPE:]).to(torch.bfloat16)
        t0 += nq
        r0 += n
    return out


# ---------------------------------------------------------------------------------------- exact results

def exact(case, seed):
    """The definition in 64 bits: per head, scores, their exponentials over the prefix, quotients."""
    st = prepare(case, seed)
    if case["op"] == "quant":
        x = st["x"].double()
        blocks = x[:, :LATENT].reshape(-1, 16)
        s = (blocks.abs().amax(1) / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
        mag = torch.tensor(GRID, dtype=torch.float64, device="cuda")
        vals = torch.empty_like(blocks)
        for i in range(0, blocks.shape[0], 1 << 16):
            u = blocks[i:i + (1 << 16)]
            si = s[i:i + (1 << 16), None]
            d = (u.abs()[..., None] - mag * si[..., None]).abs()
            # nearest magnitude; of two equally near the one whose code is even
            d = d * 2 + (torch.arange(8, device="cuda") % 2) * 1e-13 * si[..., None]
            vals[i:i + (1 << 16)] = torch.sign(u) * mag[d.argmin(-1)] * si
        return torch.cat((vals.reshape(-1, LATENT), x[:, LATENT:]), dim=1)
    H = case["heads"]
    q = st["q"].double()
    wide = HEAD_V if case["op"] == "expanded" else LATENT
    out = torch.zeros((q.shape[0], H, wide), dtype=torch.float64, device="cuda")
    lse = torch.zeros((q.shape[0], H), dtype=torch.float64, device="cuda")
    t0 = r0 = 0
    for n, nq in zip(st["lens"], st["nq"]):
        cache = st["kv"][r0:r0 + n].double() if "kv" in st else _fp4_unpack(st["kv4"][r0:r0 + n]).double()
        where = st["pos"][t0:t0 + nq].long()
        if "idx" in st:
            allow = torch.zeros((nq, n), dtype=torch.float64, device="cuda")
            for j in range(nq):
                keep = st["idx"][t0 + j]
                allow[j, keep[keep >= 0].long()] = 1
        else:
            allow = (torch.arange(n, device="cuda")[None] <= where[:, None]).double()
        for h0 in range(0, H, 1 if nq > 1 else H):
            hs = slice(h0, h0 + 1 if nq > 1 else H)
            if case["op"] == "expanded":
                for h in range(hs.start, hs.stop):
                    w = st["w_ukv"][h].double()
                    key = torch.cat((torch.einsum("sc,dc->sd", cache[:, :LATENT], w[:NOPE]), cache[:, LATENT:]), 1)
                    x = torch.einsum("td,sd->ts", q[t0:t0 + nq, h], key) * SCALE
                    top = x.masked_fill(allow == 0, -math.inf).amax(1)
                    e = torch.exp(torch.minimum(x - top[:, None], torch.zeros_like(x))) * allow
                    den = e.sum(1)
                    out[t0:t0 + nq, h] = (e @ torch.einsum("sc,dc->sd", cache[:, :LATENT], w[NOPE:])) / den[:, None]
            else:
                x = torch.einsum("thd,sd->ths", q[t0:t0 + nq, hs], cache) * SCALE
                ok = allow[:, None]
                top = x.masked_fill(ok == 0, -math.inf).amax(2)
                e = torch.exp(torch.minimum(x - top[..., None], torch.zeros_like(x))) * ok
                den = e.sum(2)
                out[t0:t0 + nq, hs] = torch.einsum("ths,sd->thd", e, cache[:, :LATENT]) / den[..., None]
                lse[t0:t0 + nq, hs] = top + torch.log(den)
        t0 += nq
        r0 += n
    return out if case["op"] == "expanded" else (out, lse)
