"""The paged 8-bit key/value cache: appends, attention, cross attention and page management.

A page holds ``page`` tokens of one sequence; a block is a page's tokens of one KV head, and its keys
and its values have one scale each.  With a = the largest magnitude in the block
  int8   code = round-half-even(127 x / a),  scale = fp32(a / 127)
  e4m3   scale = the smallest power of two with a / scale <= 448,  code = e4m3(x / scale)
and a stored entry stands for code * scale.  Attention runs on those values: softmax(scale q.k) v, causal
(query i of n sees the tokens up to L - n + i of a sequence of L) or over all of them.  Pages are taken
lowest first; a fork shares full pages and copies the last, partly filled one; compaction moves the live
pages at or beyond the live count into the free ones below it.

Kinds of cases:
  append   release the slots, append whole prompts (ragged), read the cache back as floats
  decode   one query per sequence over its cached tokens
  chunk    the last n tokens of each sequence as queries, causal
  cross    queries of a decoder over an encoder's cached states of another length, no mask
  branch   fork each sequence into several, append one token to each, decode them, free them
  compact  copy sequences to new pages, free the old ones, compact the pool, read the result and
           the page table (-1 where a sequence has no page)
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------- cases
def _case(name, kind, lens, Hq, Hkv, d, dtype, code, page, nq=None, fan=0, layers=1):
    """Lengths and query counts travel as text: a case is a dict of plain values."""
    c = {"kind": kind, "lens": " ".join(map(str, lens)), "Hq": Hq, "Hkv": Hkv, "d": d,
         "dtype": dtype, "code": code, "page": page, "nq": " ".join(map(str, nq)) if nq else "",
         "fan": fan, "layers": layers}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a batch of prompts of the 32-head model enters the cache, in lengths around the 4096-token chunk
        _case("append_prompts", "append", [4096, 5003, 4096, 2777, 6144, 4095, 4097, 2500], 32, 8, 128,
              "bf16", "int8", 64),
        # three short turns of a small model, one of a single token: launch latency counts
        _case("append_small", "append", [1, 17, 130], 4, 2, 64, "f16", "e4m3", 16),
        # a token of each of eight conversations at 32K: the library's GQA decode workload
        _case("decode_gqa32k", "decode", [32768] * 8, 32, 8, 128, "bf16", "int8", 64),
        # one user with a short context: the smallest decode
        _case("decode_one", "decode", [517], 32, 8, 128, "f16", "e4m3", 16),
        # a ragged batch in fp32, an empty and a one-token sequence in it
        _case("decode_ragged_f32", "decode", [0, 1, 15, 333, 64, 9001, 2048, 4100, 700, 77, 129, 6000],
              12, 2, 64, "f32", "int8", 32),
        # wide heads over a long document
        _case("decode_wide", "decode", [65537, 40001, 65536, 52000], 16, 4, 256, "bf16", "e4m3", 128),
        # a 64-token chunk (prompt piece or draft to check) on the 32K caches
        _case("chunk_64_on_32k", "chunk", [32768] * 8, 32, 8, 128, "bf16", "int8", 64, nq=[64] * 8),
        # two whole prompts, each attending to itself
        _case("prompt_causal", "chunk", [8192, 6001], 32, 8, 128, "bf16", "e4m3", 64, nq=[8192, 6001]),
        # decoder prefixes over encoder states of other lengths, a query head per key head
        _case("cross_prefix", "cross", [1500, 700, 1499, 250, 1, 1200, 1000, 64], 16, 16, 64, "f16", "int8",
              64, nq=[440, 33, 128, 1, 7, 300, 65, 200]),
        # one decoder token of each of 48 streams over its encoder states
        _case("cross_token", "cross", [1500 - 13 * i for i in range(48)], 16, 16, 64, "bf16", "e4m3", 32,
              nq=[1] * 48),
        # beam search: four live beams split in two and take a step
        _case("branch_beams", "branch", [1999, 1999, 2000, 2001], 32, 8, 128, "bf16", "int8", 64, fan=2),
        # long-lived pool: sequences move to new pages, the old ones are freed, the pool is compacted
        _case("compact_pool", "compact", [8192, 4100, 16000, 333, 12000, 1, 7000, 9999], 32, 8, 128, "bf16",
              "int8", 64, layers=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "chunk", "cross", "branch", "compact"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"] if kind in ("append", "decode") else ["bf16", "f16"])
    code, page = rng.choice(["int8", "e4m3"]), rng.choice([16, 32, 64, 128])
    if kind == "append":
        n = rng.randint(1, 8)
        lens = [_log(rng, 1, 6000 * 128 // d) for _ in range(n)]
        return _case("", kind, lens, Hkv, Hkv, d, dtype, code, page)
    if kind == "decode":
        n = rng.randint(1, 12)
        lens = [_log(rng, 1, 32768) if rng.random() < 0.9 else 0 for _ in range(n)]
        return _case("", kind, lens, Hkv * G, Hkv, d, dtype, code, page)
    if kind == "chunk":
        n = rng.randint(1, 4)
        nq = [_log(rng, 1, 2000) for _ in range(n)]
        lens = [q + _log(rng, 1, 6000) - 1 for q in nq]
        return _case("", kind, lens, Hkv * G, Hkv, d, dtype, code, page, nq=nq)
    if kind == "cross":
        n = rng.randint(1, 16)
        nq = [_log(rng, 1, 450) for _ in range(n)]
        lens = [_log(rng, 1, 1500) for _ in range(n)]
        return _case("", kind, lens, Hkv * G, Hkv, d, dtype, code, page, nq=nq)
    if kind == "branch":
        n = rng.randint(1, 6)
        lens = [_log(rng, 1, 8000) for _ in range(n)]
        return _case("", kind, lens, Hkv * G, Hkv, d, dtype, code, page, fan=rng.randint(1, 5))
    n = rng.randint(1, 8)
    lens = [_log(rng, 1, 10000) for _ in range(n)]
    return _case("", kind, lens, Hkv, Hkv, d, dtype, code, page, layers=rng.randint(1, 3))


def _ints(text):
    return [int(x) for x in text.split()]


def _sizes(case):
    lens = _ints(case["lens"])
    nq = _ints(case["nq"]) if case["nq"] else [1] * len(lens)
    return lens, nq


def _pages_of(lens, page):
    return [-(-n // page) for n in lens]


def work(case):
    lens, nq = _sizes(case)
    Hq, Hkv, d, page = case["Hq"], case["Hkv"], case["d"], case["page"]
    es = 4 if case["dtype"] == "f32" else 2
    tok = 2 * Hkv * d                                      # code bytes of a token
    blk = sum(_pages_of(lens, page)) * 2 * Hkv * 4         # scales
    io = 2 * Hq * d * es                                   # q and out of a query token
    kind, total = case["kind"], sum(lens)
    if kind == "append":       # floats in, codes out; codes in, floats out
        return {"bytes": 2 * (total * tok * es + total * tok + blk), "flops": 4 * total * tok}
    if kind == "decode":
        return {"bytes": total * tok + blk + len(lens) * io, "flops": 4 * d * Hq * total}
    if kind == "chunk":
        pairs = sum(n * L - n * (n - 1) // 2 for n, L in zip(nq, lens))
        return {"bytes": total * tok + blk + sum(nq) * io, "flops": 4 * d * Hq * pairs}
    if kind == "cross":
        pairs = sum(n * L for n, L in zip(nq, lens))
        return {"bytes": total * tok + blk + sum(nq) * io, "flops": 4 * d * Hq * pairs}
    if kind == "branch":       # every shared full page once, the copied partial ones per branch
        part = sum(n % page for n in lens)
        f = case["fan"]
        return {"bytes": total * tok + blk + f * part * (2 * tok + 2 * tok * es) + f * len(lens) * (io + tok * es),
                "flops": f * 4 * d * Hq * (total + len(lens))}
    # compact: copied once, moved once, read back
    pg = sum(_pages_of(lens, page)) * page
    return {"bytes": case["layers"] * (4 * pg * tok + total * tok * (1 + es)), "flops": 2 * case["layers"] * total * tok}


# ------------------------------------------------------------------------------------------- inputs
def _tokens(n, H, d, dtype, gen, spread):
    """Token-major [n, H, d]: normal entries, a few heavy channels, a norm that varies by token."""
    x = torch.randn(n, H, d, generator=gen, device="cuda")
    heavy = torch.randperm(d, generator=gen, device="cuda")[:max(1, d // 50)]
    x[..., heavy] *= 6.0
    x *= torch.exp(spread * torch.randn(n, H, 1, generator=gen, device="cuda"))
    return x.to(_DT[dtype])


def _offsets(counts):
    return torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _make(case, seed):
    """The inputs of a case, from the seed alone."""
    lens, nq = _sizes(case)
    Hq, Hkv, d, dt = case["Hq"], case["Hkv"], case["d"], case["dtype"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)
    x = {"K": [], "V": [], "lens": lens, "nq": nq}
    for _ in range(case["layers"]):
        x["K"].append(_tokens(sum(lens), Hkv, d, dt, gen, 0.2))
        x["V"].append(_tokens(sum(lens), Hkv, d, dt, gen, 0.5))
    if case["kind"] in ("decode", "chunk", "cross"):
        x["Q"] = torch.randn(sum(nq), Hq, d, generator=gen, device="cuda").to(_DT[dt])
    if case["kind"] == "branch":
        n = len(lens) * case["fan"]
        x["Q"] = torch.randn(n, Hq, d, generator=gen, device="cuda").to(_DT[dt])
        x["k1"] = _tokens(n, Hkv, d, dt, gen, 0.2)
        x["v1"] = _tokens(n, Hkv, d, dt, gen, 0.5)
    return x


def prepare(case, seed):
    lens, nq = _sizes(case)
    n, page, kind = len(lens), case["page"], case["kind"]
    x = _make(case, seed)
    npg = _pages_of(lens, page)
    st = {"case": case, "x": x, "cu": _offsets(lens), "cu_q": _offsets(nq), "max_q": max(nq),
          "slots": torch.arange(n, dtype=torch.int32, device="cuda")}
    fan = case["fan"]
    if kind == "branch":
        st["src"] = torch.arange(n * fan, dtype=torch.int32, device="cuda") // fan
        st["dst"] = torch.arange(n * fan, dtype=torch.int32, device="cuda") + n
        st["cu1"] = torch.arange(n * fan + 1, dtype=torch.int32, device="cuda")
    if kind == "compact":
        st["src"], st["dst"] = st["slots"], st["slots"] + n
    slots = n * (1 + fan) if kind == "branch" else 2 * n
    pages = 2 * sum(npg) + 2 * n * (1 + fan)
    if own:
        from compressed_attention_turboquantprod_b200 import PagedKVCache
        cache = PagedKVCache(case["Hkv"], case["d"], page=page, pages=pages, slots=slots,
                             max_pages=max(npg) + 1, code=case["code"], dtype=_DT[case["dtype"]],
                             layers=case["layers"])
        cache.extend(st["slots"], st["cu"])
        for l in range(case["layers"]):
            cache.write(x["K"][l], x["V"][l], layer=l)
        st["cache"] = cache
        return st
    # the plain cache: pages in order, padded with zeros; a table per slot
    total = sum(npg)
    first = torch.tensor([0] + npg).cumsum(0)[:-1].tolist()
    table = torch.zeros(slots, max(npg) + 1, dtype=torch.long)
    row = []
    for i in range(n):
        table[i, :npg[i]] = torch.arange(first[i], first[i] + npg[i])
        row.append(torch.arange(lens[i]) + first[i] * page)
    st["rows"] = torch.cat(row).cuda()                    # the place of each token in the pages
    st["table"] = table.cuda()
    st["lens"] = torch.tensor(lens + [0] * (slots - n)).cuda()
    st["live"] = torch.arange(pages, device="cuda") < total
    st["total"], st["pages"] = total, pages
    if kind != "append":
        st["pool"] = [[_plain_store(st, t[l], pages) for t in (x["K"], x["V"])]
                      for l in range(case["layers"])]
    return st


# ------------------------------------------------------------------------------------------- plain form
def _plain_quantise(x, code):
    """Blocks [..., page, d] -> codes, scales; 64 bits where a code is next to a rounding border."""
    a = x.float().abs().amax((-2, -1), keepdim=True)
    if code == "int8":
        ok = a >= 2.0 ** -100
        t = 127.0 * x.double() / torch.where(ok, a, 1.0).double()
        return torch.where(ok, t.round(), 0.0).to(torch.int8), torch.where(ok, a / 127.0, 0.0)[..., 0, 0]
    m, e = torch.frexp(a)
    s = torch.ldexp(torch.ones_like(a), torch.where(m <= 0.875, e - 9, e - 8))
    s = torch.where(a >= 2.0 ** -100, s, 0.0)
    y = torch.where(s > 0, x.float() / torch.where(s > 0, s, 1.0), 0.0)
    return y.to(torch.float8_e4m3fn), s[..., 0, 0]


def _plain_store(st, x, pages):
    """Token-major floats into pages: codes [pages, Hkv, page, d] and scales [pages, Hkv]."""
    case = st["case"]
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    flat = torch.zeros(st["total"] * page, Hkv, d, dtype=x.dtype, device=x.device)
    flat[st["rows"]] = x
    c, s = _plain_quantise(flat.view(st["total"], page, Hkv, d).transpose(1, 2), case["code"])
    codes = torch.zeros(pages, Hkv, page, d, dtype=c.dtype, device=c.device)
    codes.view(torch.int8)[:st["total"]] = c.view(torch.int8)
    scales = torch.zeros(pages, Hkv, device=c.device)
    scales[:st["total"]] = s
    return codes, scales


def _plain_gather(st, pool, table):
    """The floats of the pages of each row of `table`: [rows, Hkv, tokens, d]."""
    codes, scales = pool
    v = codes[table].float() * scales[table][..., None, None]        # [rows, pages, Hkv, page, d]
    r, p, h, t, d = v.shape
    return v.transpose(1, 2).reshape(r, h, p * t, d)


def _plain_attention(case, q, k, v, visible):
    """q [B, n, Hq, d]; k, v [B, Hkv, T, d]; visible [B, n]: how many tokens each query sees."""
    B, n, Hq, d = q.shape
    G = Hq // k.shape[1]
    q = q.float().view(B, n, k.shape[1], G, d).permute(0, 2, 3, 1, 4).reshape(B, k.shape[1], G * n, d)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))          # [B, Hkv, G n, T]
    hidden = torch.arange(k.shape[2], device=q.device) >= visible[:, :, None]  # [B, n, T]
    s = s.view(B, k.shape[1], G, n, -1).masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, k.shape[1], G * n, -1), v).view(B, k.shape[1], G, n, d)
    o = o / torch.where(l == 0, 1.0, l)
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, d)


def _plain_read(st, pool, table, lens):
    """The cached floats of the sequences, packed token-major [tokens, Hkv, d]."""
    v = _plain_gather(st, pool, table).transpose(1, 2)
    seen = torch.arange(v.shape[1], device=v.device) < lens[:, None]
    return v[seen].to(_DT[st["case"]["dtype"]])


def _plain_run(st):
    case, x = st["case"], st["x"]
    kind, n = case["kind"], len(x["lens"])
    width = max(1, max(_pages_of(x["lens"], case["page"])))
    if kind == "append":
        pool = [_plain_store(st, t[0], st["pages"]) for t in (x["K"], x["V"])]
        return [_plain_read(st, p, st["table"][:n, :width], st["lens"][:n]) for p in pool]
    if kind in ("decode", "chunk", "cross"):
        table, lens = st["table"][:n, :width], st["lens"][:n]
        k, v = (_plain_gather(st, p, table) for p in st["pool"][0])
        nq, mq = (st["cu_q"][1:] - st["cu_q"][:-1]).long(), st["max_q"]
        i = torch.arange(mq, device=k.device)
        real = i < nq[:, None]
        q = torch.zeros(n, mq, case["Hq"], case["d"], dtype=x["Q"].dtype, device=k.device)
        q[real] = x["Q"]
        visible = lens[:, None] - nq[:, None] + i + 1 if kind == "chunk" else lens[:, None].expand(n, mq)
        return _plain_attention(case, q, k, v, visible)[real].to(x["Q"].dtype)
    if kind == "branch":
        # full pages are shared, the last page's exact tokens and the new one are quantised anew
        src, lens, page = st["src"].long(), st["lens"][st["src"].long()], case["page"]
        full = lens // page
        b = torch.arange(len(src), device=src.device)
        out = []
        tok = torch.arange(page, device=src.device)
        at = (st["cu"][src.long()].long() + full * page)[:, None] + tok                # [B, page]
        old = tok < (lens - full * page)[:, None]
        cols = torch.arange(width + 1, device=src.device)
        for p, raw, new in zip(st["pool"][0], (x["K"][0], x["V"][0]), (x["k1"], x["v1"])):
            tail = torch.where(old[..., None, None], raw[at.clamp(max=raw.shape[0] - 1)], 0.0)
            tail[b, lens - full * page] = new
            c, s = _plain_quantise(tail.transpose(1, 2), case["code"])
            vals = _plain_gather(st, p, st["table"][src][:, :width + 1])
            r, h, _, d = vals.shape
            vals = vals.view(r, h, width + 1, page, d)
            last = (cols == full[:, None])[:, None, :, None, None]
            out.append(torch.where(last, (c.float() * s[..., None, None])[:, :, None], vals)
                       .view(r, h, (width + 1) * page, d))
        return _plain_attention(case, x["Q"][:, None], out[0], out[1], lens[:, None] + 1)[:, 0].to(x["Q"].dtype)
    # compact: copy to the lowest free pages, free the first ones, move the live pages down
    src, lens = st["src"].long(), torch.tensor(x["lens"], device="cuda")
    used = torch.arange(st["table"].shape[1], device="cuda") < -(-lens // case["page"])[:, None]
    old = st["table"][:n][used]
    free = torch.nonzero(~st["live"])[:len(old), 0]
    live = st["live"].clone()
    live[free], live[old] = True, False
    count = int(len(old))
    holes = torch.nonzero(~live[:count])[:, 0]
    moved = count + torch.nonzero(live[count:])[:, 0]
    to = torch.arange(st["pages"], device="cuda")
    to[moved] = holes
    table = torch.zeros_like(st["table"][:n])
    table[used] = to[free]
    out = []
    for pools in st["pool"]:
        for codes, scales in pools:
            c, s = codes.view(torch.int8), scales
            c[free], s[free] = c[old], s[old]
            c[holes], s[holes] = c[moved], s[moved]
            out.append(_plain_read(st, (codes, scales), table[:, :width], lens))
    return out + [torch.where(used, table, -1)]


# ------------------------------------------------------------------------------------------- a pass
def run(state):
    if not own:
        return _plain_run(state)
    case, x, cache = state["case"], state["x"], state["cache"]
    kind = case["kind"]
    if kind == "append":
        cache.free(state["slots"])
        cache.append(x["K"][0], x["V"][0], state["slots"], state["cu"])
        return cache.read(state["slots"], state["cu"], x["K"][0].shape[0])
    if kind == "decode":
        return cache.decode(x["Q"], state["slots"])
    if kind == "chunk":
        return cache.attend(x["Q"], state["slots"], state["cu_q"], state["max_q"])
    if kind == "cross":
        return cache.cross(x["Q"], state["slots"], state["cu_q"], state["max_q"])
    if kind == "branch":
        cache.fork(state["src"], state["dst"])
        out = cache.decode_step(x["k1"], x["v1"], x["Q"], state["dst"], state["cu1"])
        cache.free(state["dst"])
        return out
    src, dst = state["src"], state["dst"]
    cache.copy(src, dst)
    cache.free(src)
    cache.compact()
    out = []
    for l in range(case["layers"]):
        out += cache.read(dst, state["cu"], x["K"][l].shape[0], layer=l)
    state["src"], state["dst"] = dst, src            # the next pass takes them back
    return out + [cache.page_table(dst).long()]


# ------------------------------------------------------------------------------------------- 64 bits
def _exact_block(x, code):
    """The values a block [tokens, d] stands for, in float64."""
    x = x.double()
    a = float(x.abs().max())
    if a < 2.0 ** -100:
        return torch.zeros_like(x)
    if code == "int8":
        return torch.round(127.0 * x / a) * (a / 127.0)
    s = 2.0 ** math.ceil(math.log2(a / 448.0))
    y = x / s
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * s


def _exact_cached(x, code, page):
    """One sequence's tokens [T, H, d] as the cache holds them, in float64."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    T = x.shape[0]
    whole = T // page * page
    if whole:
        y = x[:whole].double().view(-1, page, x.shape[1], x.shape[2])
        a = y.abs().amax((1, 3), keepdim=True)
        if code == "int8":
            z = torch.round(127.0 * y / a.clamp(min=2.0 ** -100)) * (a / 127.0)
        else:
            k = torch.ceil(torch.log2(a.clamp(min=2.0 ** -100) / 448.0))
            w = y / torch.exp2(k)
            step = torch.exp2(torch.floor(torch.log2(w.abs().clamp(min=2.0 ** -6))) - 3)
            z = torch.round(w / step) * step * torch.exp2(k)
        out[:whole] = torch.where(a < 2.0 ** -100, 0.0, z).reshape(whole, x.shape[1], x.shape[2])
    for h in range(x.shape[1] if T > whole else 0):
        out[whole:, h] = _exact_block(x[whole:, h], code)
    return out


def _exact_attention(q, k, v, offset):
    """q [n, Hq, d] over k, v [T, Hkv, d] (float64); query i sees tokens t <= offset + i (None: all)."""
    n, Hq, d = q.shape
    T, Hkv, _ = k.shape
    out = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device)
    if T == 0:
        return out
    G = Hq // Hkv
    for lo in range(0, n, 1024):
        hi = min(n, lo + 1024)
        end = T if offset is None else max(0, min(T, offset + hi))
        if end == 0:
            continue
        for h in range(Hkv):
            s = torch.einsum("ngd,td->gnt", q[lo:hi, h * G:(h + 1) * G].double(), k[:end, h]) / math.sqrt(d)
            if offset is not None:
                seen = torch.arange(end, device=q.device)[None] <= (torch.arange(lo, hi, device=q.device) + offset)[:, None]
                s = s.masked_fill(~seen, float("-inf"))
            p = torch.nan_to_num(torch.softmax(s, -1))
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", p, v[:end, h])
    return out


def exact(case, seed):
    x = _make(case, seed)
    lens, nq, code, page, kind = x["lens"], x["nq"], case["code"], case["page"], case["kind"]
    starts = [sum(lens[:i]) for i in range(len(lens))]

    def cached(t, i):
        return _exact_cached(t[starts[i]:starts[i] + lens[i]], code, page)

    if kind in ("append", "compact"):
        out = []
        for l in range(case["layers"]):
            for t in (x["K"][l], x["V"][l]):
                out.append(torch.cat([cached(t, i) for i in range(len(lens))]))
        return out if kind == "append" else out + [None]
    res, at = [], 0
    for i, L in enumerate(lens):
        if kind == "branch":
            for f in range(case["fan"]):
                b = i * case["fan"] + f
                k, v = (_exact_cached(torch.cat([t[starts[i]:starts[i] + L], y[b:b + 1]]), code, page)
                        for t, y in ((x["K"][0], x["k1"]), (x["V"][0], x["v1"])))
                res.append(_exact_attention(x["Q"][b:b + 1], k, v, None))
            continue
        k, v = cached(x["K"][0], i), cached(x["V"][0], i)
        res.append(_exact_attention(x["Q"][at:at + nq[i]], k, v, L - nq[i] if kind == "chunk" else None))
        at += nq[i]
    return torch.cat(res)
