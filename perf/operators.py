"""Three operators over the compressed KV cache, in their plain form and as calls of the library.

  read_back      nsn_dequantize_kv: the tokens of a compressed cache as ordinary rows.
  decode_prefix  nsn_decode_attention_prefix: one new token per sequence, attention over a
                 compressed prefix that the whole batch shares and over each sequence's own cache.
  extend_prefix  nsn_extend_attention_prefix: the same for a chunk of new tokens per sequence,
                 causal inside the chunk.

A cached token is x_hat = H^T ((u_hat s2 + o) s1): u_hat the codewords of its 16 codes (with the
stored signs in 2-bit mode, entries rounded to fp16), s1 and s2 its two norms, o the mean of its
128-token block, H the orthonormal Hadamard matrix.  Window tokens are stored as they are.
"""
import math
import random

import torch

own = False

D, SUB, NSUB, NCODES, BLK = 128, 8, 16, 256, 128
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a 256-token 1-bit cache read back whole: latency
        _read_back("read_256_1bit_f32", batch=1, heads=1, tokens=256, window=0, mode=1, dtype="float32"),
        # one layer's prompt cache handed to a full-precision consumer
        _read_back("read_4096_2bit_bf16", batch=1, heads=8, tokens=4096, window=128, mode=2, dtype="bfloat16"),
        # the later part of a ragged batch, double quantization, head-major output, odd start
        _read_back("read_ragged_dq_f16", batch=16, heads=8, tokens=5003, window=128, mode=2, dtype="float16", dq=True,
                   start=1001, ragged=True, heads_first=True),
        # every token of a 16 x 32k layer, as when a cache is moved to another engine
        _read_back("read_16x32768_2bit_bf16", batch=16, heads=8, tokens=32768, window=128, mode=2, dtype="bfloat16"),
        # a few samples of one prompt: latency of a small call
        _attend("decode_4_prefix_4096", batch=4, chunk=0, prefix=4096, suffix=100, mode_k=2, mode_v=2),
        # an odd batch of fp16 queries over a prefix that ends inside a block, 8 queries per kv-head, double quantization
        _attend("decode_7_prefix_1000_dq", batch=7, chunk=0, heads=2, group=8, prefix=1000, prefix_window=0, suffix=333,
                mode_k=2, mode_v=1, dq=True, dtype="float16", ragged=True),
        # a serving batch behind a 32k system prompt
        _attend("decode_16_prefix_32768", batch=16, chunk=0, prefix=32768, suffix=300, mode_k=2, mode_v=2, ragged=True),
        # the 64-sequence batch over a long shared context, mixed 2-bit K / 1-bit V
        _attend("decode_64_prefix_131072", batch=64, chunk=0, prefix=131072, suffix=200, mode_k=2, mode_v=1, ragged=True),
        # a few speculated tokens per sequence
        _attend("extend_4x5_prefix_4096", batch=4, chunk=5, prefix=4096, suffix=60, mode_k=2, mode_v=2),
        # odd sizes: a 33-token chunk, 1-bit cache, 2 queries per kv-head, fp16
        _attend("extend_3x33_prefix_2500_1bit", batch=3, chunk=33, heads=4, group=2, prefix=2500, suffix=700, mode_k=1,
                mode_v=1, dtype="float16", ragged=True),
        # a chunk of a user's prompt behind a cached document
        _attend("extend_4x128_prefix_8192", batch=4, chunk=128, prefix=8192, suffix=1500, mode_k=2, mode_v=2, ragged=True),
        # the same for a batch of 8 behind a 32k prompt: the largest
        _attend("extend_8x128_prefix_32768", batch=8, chunk=128, prefix=32768, suffix=600, mode_k=2, mode_v=2, ragged=True),
    ]


def _read_back(name, batch, heads, tokens, window, mode, dtype, dq=False, start=0, ragged=False, heads_first=False):
    return {"name": name, "op": "read_back", "batch": batch, "heads": heads, "tokens": tokens, "window": window, "mode": mode,
            "dtype": dtype, "dq": dq, "start": start, "ragged": ragged, "heads_first": heads_first}


def _attend(name, batch, chunk, prefix, suffix, mode_k, mode_v, heads=8, group=4, prefix_window=128, dq=False,
            dtype="bfloat16", ragged=False):
    """chunk 0: decode of one token per sequence; otherwise that many new tokens, the last ones of each sequence."""
    return {"name": name, "op": "extend_prefix" if chunk else "decode_prefix", "batch": batch, "chunk": chunk, "heads": heads,
            "group": group, "prefix": prefix, "prefix_window": prefix_window, "suffix": suffix, "mode_k": mode_k,
            "mode_v": mode_v, "dq": dq, "dtype": dtype, "ragged": ragged}


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["read_back", "decode_prefix", "extend_prefix"])
    if op == "read_back":
        batch, heads = _spread(rng, 1, 16), rng.choice([1, 2, 5, 8])
        tokens = _spread(rng, 1, 16384)
        case = _read_back("", batch, heads, tokens, rng.choice([0, 128]), rng.choice([1, 2]), rng.choice(list(DTYPES)),
                          dq=rng.random() < 0.3, start=rng.choice([0, rng.randrange(tokens)]), ragged=rng.random() < 0.5,
                          heads_first=rng.random() < 0.3)
    else:
        chunk = 0 if op == "decode_prefix" else _spread(rng, 1, 128)
        batch = _spread(rng, 1, 8 if chunk else 64)
        case = _attend("", batch, chunk, prefix=_spread(rng, 1, 30000 if chunk else 65536), suffix=_spread(rng, max(1, chunk), 1500),
                       mode_k=rng.choice([1, 2]), mode_v=rng.choice([1, 2]), heads=rng.choice([1, 2, 5, 8]),
                       group=rng.choice([1, 2, 4, 4, 8]) if batch * max(chunk, 1) <= 512 else rng.choice([1, 2, 4]),
                       prefix_window=rng.choice([0, 128]), dq=rng.random() < 0.3, dtype=rng.choice(["bfloat16", "float16"]),
                       ragged=rng.random() < 0.5)
    del case["name"]
    return case


def _lengths(batch, most, least, ragged):
    """Tokens of each sequence: `most`, or spread below it (never under `least`)."""
    span = most - least + 1
    return [most - (b * 7919) % span if ragged else most for b in range(batch)]


def _suffixes(case):
    """Tokens of each sequence's own cache: a chunk sits whole in the window, so it ends with that many window tokens."""
    chunk = max(case["chunk"], 1)
    lengths = _lengths(case["batch"], case["suffix"], chunk, case["ragged"])
    return [n if _split(n, BLK)[1] >= chunk else n - n % BLK for n in lengths]


def _split(n, window):
    """(quantized, window) tokens of a sequence of n: the last 1..128 stay in the window, where there is one."""
    quantized = n if window == 0 else BLK * ((n - 1) // BLK) if n else 0
    return quantized, n - quantized


# ---------------------------------------------------------------------------
# Inputs: keys and values with outlier channels, quantized here with plain torch operations
# ---------------------------------------------------------------------------
def _hadamard(dtype, device):
    h = torch.ones((1, 1), dtype=dtype, device=device)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(D)


def _codebook(gen, mode):
    """256 codewords of 8 values: a few rounds of k-means on normal samples (their absolute values in 2-bit mode)."""
    x = torch.randn((8192, SUB), generator=gen, device="cuda")
    x = x.abs() if mode == 2 else x
    c = x[:NCODES].clone()
    for _ in range(8):
        near = (x @ c.t() - 0.5 * (c * c).sum(1)).argmax(1)
        member = (near[:, None] == torch.arange(NCODES, device="cuda")).float()
        count = member.sum(0)
        c = torch.where(count[:, None] > 0, (member.t() @ x) / count.clamp(min=1)[:, None], c)
    return c.half().float()


def _tokens(gen, batch, heads, n):
    """[batch, heads, n, 128] in bf16: normal, with five outlier channels per head."""
    x = torch.randn((batch, heads, n, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    order = torch.rand((heads, D), generator=gen, device="cuda").argsort(1)[:, :5]
    scale = torch.ones((heads, D), device="cuda").scatter_(1, order, 3.0)
    shift = torch.zeros((heads, D), device="cuda").scatter_(1, order, 12.0 * torch.randn((heads, 5), generator=gen, device="cuda"))
    return x.mul_(scale[:, None].bfloat16()).add_(shift[:, None].bfloat16())


def _levels(x, dim):
    """Sixteen uniform levels between the fp16 ends of a group: (levels, lo, hi)."""
    lo, hi = x.amin(dim, keepdim=True).half(), x.amax(dim, keepdim=True).half()
    step = (hi.float() - lo.float()) / 15
    lev = torch.where(step > 0, (x - lo.float()) / step.clamp(min=1e-20), torch.zeros_like(x)).round().clamp(0, 15)
    return lev.to(torch.uint8), lo, hi


def _fill(cache, rows, lengths, codebook, mode, dq, window):
    """Quantizes rows [B, H, n, 128] into the buffers of `cache`, sequence b with its first lengths[b] tokens."""
    had = _hadamard(torch.float32, "cuda")
    heads = rows.shape[1]
    for b, n in enumerate(lengths):
        nq, nw = _split(n, window)
        cache["n_quant"][b], cache["n_window"][b] = nq, nw
        if nw:
            cache["window"][b, :, :nw] = rows[b, :, nq:n].half()
        for t0 in range(0, nq, 16384):
            t1 = min(nq, t0 + 16384)
            m, nb = t1 - t0, (t1 - t0 + BLK - 1) // BLK
            y = torch.zeros((heads, nb * BLK, D), device="cuda")
            y[:, :m] = rows[b, :, t0:t1].float() @ had.t()
            y = y.view(heads, nb, BLK, D)
            here = (torch.arange(nb * BLK, device="cuda") < m).view(1, nb, BLK, 1)
            s1 = y.square().mean(-1, keepdim=True).sqrt()
            n1 = y / s1.clamp(min=1e-20)
            o = n1.sum(2, keepdim=True) / here.sum(2, keepdim=True)
            z = torch.where(here, n1 - o, torch.zeros_like(n1))
            s2 = z.square().mean(-1, keepdim=True).sqrt()
            u = (z / s2.clamp(min=1e-20)).reshape(-1, NSUB, SUB)
            a = u.abs() if mode == 2 else u
            code = torch.cat([(part @ codebook.t() - 0.5 * codebook.square().sum(1)).argmax(-1) for part in a.split(16384)])
            hat = codebook[code] * (torch.where(u < 0, -1.0, 1.0) if mode == 2 else 1.0)
            dot = (u * hat).sum((1, 2))
            alpha = torch.where(dot > 0, u.square().sum((1, 2)) / dot.clamp(min=1e-20), torch.ones_like(dot)).view(s2.shape)
            code = code.view(heads, -1, NSUB)[:, :m].to(torch.uint8)
            cache["codes"][b, :, t0:t1] = torch.cat([code[..., 0::2], code[..., 1::2]], -1)
            if mode == 2:
                bits = (u.view(heads, -1, NSUB, SUB)[:, :m] < 0).int() << (15 - torch.arange(NSUB, device="cuda", dtype=torch.int32))[:, None]
                field = bits.sum(2)                                                   # [heads, m, 8]
                cache["signs"][b, :, t0:t1] = torch.stack([field & 255, field >> 8], -1).flatten(-2).to(torch.uint8)
            first, last = t0 // BLK, t0 // BLK + nb
            s1, s2 = s1.reshape(heads, nb, BLK), (alpha * s2).reshape(heads, nb * BLK)[:, :m]
            if dq:
                least = torch.where(here[..., 0], s1, s1[..., :1])                    # rows past the end repeat the first
                lev, lo, hi = _levels(least, 2)
                lev = lev.reshape(heads, nb * BLK)
                cache["s1_levels"][b, :, t0 // 2:t0 // 2 + nb * BLK // 2] = lev[:, 0::2] | (lev[:, 1::2] << 4)
                olev, olo, ohi = _levels(o[:, :, 0], 2)
                cache["means"][b, :, first:last] = olev[..., 0::2] | (olev[..., 1::2] << 4)
                cache["dq_params"][b, :, first:last, :4] = torch.cat([lo, hi, olo, ohi], -1)
                cache["norms"][b, :, t0:t1] = s2.half()
            else:
                cache["norms"][b, :, t0:t1] = torch.stack([s1.reshape(heads, nb * BLK)[:, :m], s2], -1).half()
                cache["means"][b, :, first:last] = o[:, :, 0].half()
    return cache


def _empty(batch, heads, capacity, window, mode, dq):
    """The buffers of one compressed cache, in the library's layout."""
    z = lambda shape, dt: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
    nb = capacity // BLK
    return {"codes": z((batch, heads, capacity, NSUB), torch.uint8),
            "signs": z((batch, heads, capacity, NSUB), torch.uint8) if mode == 2 else None,
            "norms": z((batch, heads, capacity) if dq else (batch, heads, capacity, 2), torch.float16),
            "means": z((batch, heads, nb, D // 2), torch.uint8) if dq else z((batch, heads, nb, D), torch.float16),
            "s1_levels": z((batch, heads, capacity // 2), torch.uint8) if dq else None,
            "dq_params": z((batch, heads, nb, 8), torch.float16) if dq else None,
            "window": z((batch, heads, window, D), torch.float16) if window else None,
            "n_quant": z((batch, heads), torch.int32), "n_window": z((batch, heads), torch.int32)}


def _cache(gen, batch, heads, lengths, window, mode, dq, codebook):
    capacity = BLK * max(1, -(-max(lengths) // BLK))
    rows = _tokens(gen, batch, heads, max(lengths))
    return _fill(_empty(batch, heads, capacity, window, mode, dq), rows, lengths, codebook, mode, dq, window)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "read_back":
        lengths = _lengths(case["batch"], case["tokens"], 1, case["ragged"])
        cb = _codebook(gen, case["mode"])
        cache = _cache(gen, case["batch"], case["heads"], lengths, case["window"], case["mode"], case["dq"], cb)
        n = case["tokens"] - case["start"]
        shape = (case["batch"], case["heads"], n, D) if case["heads_first"] else (case["batch"], n, case["heads"], D)
        out = torch.zeros(shape, dtype=DTYPES[case["dtype"]], device="cuda")
        return {"cache": cache, "cb": cb, "out": out.transpose(1, 2) if case["heads_first"] else out}
    chunk, heads, dq = max(case["chunk"], 1), case["heads"], case["dq"]
    cbk, cbv = _codebook(gen, case["mode_k"]), _codebook(gen, case["mode_v"])
    lengths = _suffixes(case)
    make = lambda batch, n, window, mode, cb: _cache(gen, batch, heads, n, window, mode, dq, cb)  # noqa: E731
    n_q = heads * case["group"]
    shape = (case["batch"], case["chunk"], n_q, D) if case["chunk"] else (case["batch"], n_q, D)
    dt = DTYPES[case["dtype"]]
    return {"pk": make(1, [case["prefix"]], case["prefix_window"], case["mode_k"], cbk),
            "pv": make(1, [case["prefix"]], case["prefix_window"], case["mode_v"], cbv),
            "k": make(case["batch"], lengths, BLK, case["mode_k"], cbk),
            "v": make(case["batch"], lengths, BLK, case["mode_v"], cbv),
            "cbk": cbk, "cbv": cbv, "q": torch.randn(shape, generator=gen, device="cuda").to(dt),
            "out": torch.zeros(shape, dtype=dt, device="cuda")}


def _handle(buffers, window, mode, dq):
    """The library's cache with these contents."""
    from calibration_free_vector_b200 import nsn
    batch, heads, capacity = buffers["codes"].shape[:3]
    c = nsn.Cache(batch, heads, capacity, window, mode, double_quant=dq)
    for mine, theirs in (("codes", "codes"), ("signs", "signs"), ("norms", "norms"), ("means", "means"),
                         ("s1_levels", "s1_levels"), ("dq_params", "dq_params"), ("window", "window_buf"),
                         ("n_quant", "n_quant"), ("n_window", "n_window")):
        if buffers[mine] is not None:
            getattr(c, theirs).copy_(buffers[mine])
    return c


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if own:
        from calibration_free_vector_b200 import nsn
        if case["op"] == "read_back":
            s["cache"] = _handle(s["cache"], case["window"], case["mode"], case["dq"])
        else:
            for name, window, mode in (("pk", case["prefix_window"], case["mode_k"]), ("pv", case["prefix_window"], case["mode_v"]),
                                       ("k", BLK, case["mode_k"]), ("v", BLK, case["mode_v"])):
                s[name] = _handle(s[name], window, mode, case["dq"])
            s["workspace"] = nsn.prefix_workspace(s["pk"], s["k"], case["heads"] * case["group"], max(case["chunk"], 1))
    return s


# ---------------------------------------------------------------------------
# The operators: the library's calls, and their plain form in 32 bits
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        from calibration_free_vector_b200 import nsn
        if case["op"] == "read_back":
            nsn.nsn_dequantize_kv(s["cache"], s["out"], s["cb"], start=case["start"])
        else:
            call = nsn.nsn_extend_attention_prefix if case["chunk"] else nsn.nsn_decode_attention_prefix
            call(s["pk"], s["pv"], s["k"], s["v"], s["q"], 1 / math.sqrt(D), s["cbk"], s["cbv"], s["out"], s["workspace"])
        return s["out"]
    if case["op"] == "read_back":
        return _plain_read_back(s)
    return _plain_attend(s)


def _plain_rows(c, cb):
    """The quantized part of a cache as fp32 rows [B, H, capacity, 128]."""
    code = torch.stack([c["codes"][..., :8], c["codes"][..., 8:]], -1).flatten(-2).long()
    u = cb.half().float()[code]                                                       # [B, H, T, 16, 8]
    if c["signs"] is not None:
        field = c["signs"].view(torch.int16).int()[..., None, :]                      # [B, H, T, 1, 8]
        bit = (field >> (15 - torch.arange(NSUB, device=u.device, dtype=torch.int32))[:, None]) & 1
        u = u * (1 - 2 * bit)
    if c["dq_params"] is None:
        s1, s2, o = c["norms"][..., 0].float(), c["norms"][..., 1].float(), c["means"].float()
    else:
        par = c["dq_params"].float()
        lev = torch.stack([c["s1_levels"] & 15, c["s1_levels"] >> 4], -1).flatten(-2).float()
        lev = lev.unflatten(-1, (-1, BLK))
        s1 = (par[..., 0:1] + lev * ((par[..., 1:2] - par[..., 0:1]) / 15)).flatten(-2)
        olev = torch.stack([c["means"] & 15, c["means"] >> 4], -1).flatten(-2).float()
        o = par[..., 2:3] + olev * ((par[..., 3:4] - par[..., 2:3]) / 15)
        s2 = c["norms"].float()
    z = u.flatten(-2).unflatten(-2, (-1, BLK)) * s2.unflatten(-1, (-1, BLK))[..., None] + o[..., None, :]
    return (z.flatten(-3, -2) * s1[..., None]) @ _hadamard(torch.float32, z.device)


def _plain_read_back(s):
    c, start, n = s["cache"], s["case"]["start"], s["out"].shape[1]
    rows = _plain_rows(c, s["cb"])
    t = start + torch.arange(n, device=rows.device)
    nq, total = c["n_quant"][..., None], (c["n_quant"] + c["n_window"])[..., None]
    x = rows[:, :, t.clamp(max=rows.shape[2] - 1)]
    if c["window"] is not None:
        slot = (t - nq).clamp(0, BLK - 1).long()
        x = torch.where((t < nq)[..., None], x, c["window"].float().gather(2, slot[..., None].expand(-1, -1, -1, D)))
    return torch.where((t < total)[..., None].transpose(1, 2), x.transpose(1, 2).to(s["out"].dtype), s["out"])


def _plain_side(c, cb, chunk):
    """Rows of a cache with its window, and which of them each of the chunk's tokens sees: [B, H, chunk, tokens]."""
    rows = _plain_rows(c, cb)
    t = torch.arange(rows.shape[2], device=rows.device)
    seen = (t < c["n_quant"][..., None])[:, :, None].expand(-1, -1, chunk, -1)
    if c["window"] is not None:
        rows = torch.cat([rows, c["window"].float()], 2)
        last = c["n_window"][..., None] - chunk + 1 + torch.arange(chunk, device=rows.device)
        seen = torch.cat([seen, torch.arange(BLK, device=rows.device) < last[..., None]], -1)
    return rows, seen


def _plain_attend(s):
    case = s["case"]
    chunk, heads, group = max(case["chunk"], 1), case["heads"], case["group"]
    q = s["q"].float().view(case["batch"], chunk, heads, group, D) / math.sqrt(D)
    (pk, seen_p), (pv, _) = _plain_side(s["pk"], s["cbk"], 1), _plain_side(s["pv"], s["cbv"], 1)
    (k, seen), (v, _) = _plain_side(s["k"], s["cbk"], chunk), _plain_side(s["v"], s["cbv"], chunk)
    low = torch.full((), -math.inf, device=q.device)
    sp = torch.where(seen_p[0, :, 0], torch.einsum("bchgd,htd->bcght", q, pk[0]), low)
    so = torch.where(seen.permute(0, 2, 1, 3)[:, :, None], torch.einsum("bchgd,bhtd->bcght", q, k), low)
    top = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True)).clamp(min=-1e30)
    ep, eo = (sp - top).exp_(), (so - top).exp_()
    total = ep.sum(-1) + eo.sum(-1)
    x = torch.einsum("bcght,htd->bcghd", ep, pv[0]) + torch.einsum("bcght,bhtd->bcghd", eo, v)
    x = x / total.clamp(min=1e-30)[..., None]
    return x.permute(0, 1, 3, 2, 4).reshape(s["out"].shape).to(s["out"].dtype)


# ---------------------------------------------------------------------------
# The definition in 64 bits, one head at a time
# ---------------------------------------------------------------------------
def _exact_rows(c, cb, b, h):
    """Every token of one sequence in order, quantized ones first: [n, 128] in fp64."""
    n, nw = int(c["n_quant"][b, h]), int(c["n_window"][b, h])
    table = cb.to(torch.float16).double()
    y = torch.empty((n, D), dtype=torch.float64, device=cb.device)
    for sub in range(NSUB):
        code = c["codes"][b, h, :n, (sub // 2) + (8 if sub % 2 else 0)].long()
        y[:, SUB * sub:SUB * sub + SUB] = table[code]
    if c["signs"] is not None:
        for i in range(SUB):
            word = c["signs"][b, h, :n, 2 * i].int() + 256 * c["signs"][b, h, :n, 2 * i + 1].int()
            for sub in range(NSUB):
                y[:, SUB * sub + i] *= torch.where((word & (1 << (15 - sub))) != 0, -1.0, 1.0).double()
    block = torch.arange(n, device=cb.device) // BLK
    if c["dq_params"] is None:
        s1, s2, o = c["norms"][b, h, :n, 0].double(), c["norms"][b, h, :n, 1].double(), c["means"][b, h].double()
    else:
        lo1, hi1, lo, hi = (c["dq_params"][b, h, :, i].double() for i in range(4))
        packed = c["s1_levels"][b, h, torch.arange(n, device=cb.device) // 2].int()
        lev = torch.where(torch.arange(n, device=cb.device) % 2 == 1, packed // 16, packed % 16).double()
        s1 = lo1[block] + lev * (hi1 - lo1)[block] / 15
        s2 = c["norms"][b, h, :n].double()
        o = torch.empty((c["means"].shape[2], D), dtype=torch.float64, device=cb.device)
        o[:, 0::2], o[:, 1::2] = (c["means"][b, h] % 16).double(), (c["means"][b, h] // 16).double()
        o = lo[:, None] + o * (hi - lo)[:, None] / 15
    y = (y * s2[:, None] + o[block]) * s1[:, None]
    width = 1
    while width < D:                                                                  # butterflies: the Hadamard transform
        y = y.view(n, D // (2 * width), 2, width)
        y = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(n, D)
        width *= 2
    y = y / math.sqrt(D)
    return torch.cat([y, c["window"][b, h, :nw].double()]) if nw else y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "read_back":
        out = s["out"].double()
        for b in range(case["batch"]):
            for h in range(case["heads"]):
                x = _exact_rows(s["cache"], s["cb"], b, h)[case["start"]:]
                out[b, :len(x), h] = x
        return out
    chunk, group = max(case["chunk"], 1), case["group"]
    q = s["q"].double().view(case["batch"], chunk, case["heads"], group, D)
    out = torch.zeros_like(q)
    for h in range(case["heads"]):
        pk, pv = _exact_rows(s["pk"], s["cbk"], 0, h), _exact_rows(s["pv"], s["cbv"], 0, h)
        for b in range(case["batch"]):
            k = torch.cat([pk, _exact_rows(s["k"], s["cbk"], b, h)])
            v = torch.cat([pv, _exact_rows(s["v"], s["cbv"], b, h)])
            score = (q[b, :, h].reshape(-1, D) @ k.t() / math.sqrt(D)).view(chunk, group, -1)
            for i in range(chunk - 1):
                score[i, :, score.shape[-1] - chunk + 1 + i:] = -math.inf
            out[b, :, h] = torch.softmax(score, -1) @ v
    return out.view(s["q"].shape)


# ---------------------------------------------------------------------------
# Work
# ---------------------------------------------------------------------------
def _stored(n, window, mode, dq):
    """Bytes of one head's n cached tokens."""
    nq, nw = _split(n, window)
    blocks = -(-nq // BLK)
    return nq * (NSUB * mode + (2.5 if dq else 4)) + blocks * (D // 2 + 16 if dq else 2 * D) + nw * 2 * D


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "read_back":
        lengths = _lengths(case["batch"], case["tokens"], 1, case["ragged"])
        rows = sum(max(0, n - case["start"]) for n in lengths) * case["heads"]
        per_token = _stored(BLK * 64, 0, case["mode"], case["dq"]) / (BLK * 64)
        # a token: its record read, its row written; the transform's 7 x 128 additions, scale and mean
        return {"bytes": rows * (per_token + D * size), "flops": rows * D * 11}
    chunk = max(case["chunk"], 1)
    lengths = _suffixes(case)
    stored = sum(_stored(case["prefix"], case["prefix_window"], m, case["dq"]) + sum(_stored(n, BLK, m, case["dq"]) for n in lengths)
                 for m in (case["mode_k"], case["mode_v"])) * case["heads"]
    rows = case["batch"] * chunk * case["heads"] * case["group"]
    pairs = rows * case["prefix"] + sum(n - (chunk - 1) / 2 for n in lengths) * chunk * case["heads"] * case["group"]
    return {"bytes": stored + 2 * rows * D * size, "flops": 4 * D * pairs}


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(c.get("name", "drawn"), work(c))
