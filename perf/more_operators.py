"""The 4-bit cache operators' work cases: inputs, plain forms, exact values and costs.

Five kinds of call: "store" (new keys and values of several sequences rounded to 4 bits into
their pages, and read back as the values the cache stands for from then on), "attend" (queries
against such a cache: single tokens, a few of a draft, long pieces of a prompt), "fork" (sequences
that go on from others: shared pages, copies of those written in part, pages for the next tokens,
pages given back), "compact" (the pages in use moved to the front of the pool) and "copy" (listed
pages to another pool).

The cache.  A pool is bytes [pages][page bytes]; a page holds `page` tokens of every key head, a
head's tokens in strips of 16.  Values are rounded in blocks of 32 channels of one token and head
(the last one of a head may be shorter): a power of two 2^e, held in 8 bits as e + 127, and for
each value a sign and one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.  e is the smallest exponent
for which the largest magnitude of the block is at most 7 * 2^e; values are rounded to the nearest,
ties to the even code.  With n blocks a head, a strip is
    keys        [4 groups g][16 tokens][n blocks][4 bytes b]   channels 8 g + 2 b, + 1 of the block
    values      [4 groups g][16 pairs r][n blocks][4 tokens]   tokens 4 g + i, channels 2 r, 2 r + 1
    keys' e     [16 tokens][n, or 4 where n is 3]
    values' e   [4 groups g][n blocks][4 tokens]
the first of two channels in the lower half of a byte.  A table's row lists a sequence's pages, -1
where there is none; owners[p] counts the entries (and other holds) of page p.

`own` false: elementary torch operations; `own` true: the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EXPONENTS = {"f32": (-120, 125), "bf16": (-120, 125), "f16": (-23, 13)}
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BORDERS = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]     # to the even code: the 2nd, 4th, 6th go up


def _ints(text):
    return [int(v) for v in text.split(",")]


def _strip_bytes(dim):
    n = -(-dim // 32)
    return 16 * (32 * n + (4 if n == 3 else n) + n)


def _page_bytes(case):
    return _strip_bytes(case["dim"]) * case["heads"] * case["page"] // 16


# ------------------------------------------------------------------ the cases

def _named(name, case):
    return dict(case, name=name) if name else case


def _store(name, dtype, lens, new, heads, dim, page):
    return _named(name, dict(op="store", dtype=dtype, lens=lens, new=new, heads=heads, dim=dim,
                             page=page))


def _attend(name, dtype, lens, new, q_heads, heads, dim, page, causal=True):
    return _named(name, dict(op="attend", dtype=dtype, lens=lens, new=new, q_heads=q_heads,
                             heads=heads, dim=dim, page=page, causal=causal))


def _fork(name, lens, beams, kept, layers, heads, dim, page):
    return _named(name, dict(op="fork", lens=lens, beams=beams, kept=kept, layers=layers,
                             heads=heads, dim=dim, page=page))


def _compact(name, pages, live, rows, layers, heads, dim, page):
    return _named(name, dict(op="compact", pages=pages, live=live, rows=rows, layers=layers,
                             heads=heads, dim=dim, page=page))


def _copy(name, pages, count, layers, heads, dim, page):
    return _named(name, dict(op="copy", pages=pages, count=count, layers=layers, heads=heads,
                             dim=dim, page=page))


def listed():
    return [
        # the new token of each of a serving batch of 48
        _store("store step bf16", "bf16", ",".join(str(1 + (i * 613 + 11) % 4096) for i in range(48)),
               ",".join(["1"] * 48), 8, 128, 16),
        # prompts of very different lengths at full precision, one of them a piece behind earlier
        # tokens, a head size between the usual ones
        _store("store prompts f32", "f32", "4096,1,1337,2048,700,9", "4096,1,1337,1001,700,9", 8, 80, 64),
        # one new token after a prompt of one user: latency
        _attend("attend step f16", "f16", "4097", "1", 32, 8, 128, 16),
        # a serving batch of 48 with between 1 and 16384 tokens in its caches
        _attend("attend batch bf16", "bf16",
                ",".join(str(1 + (i * 6151 + 11) % 16384) for i in range(48)),
                ",".join(["1"] * 48), 32, 8, 128, 16),
        # drafts of five tokens at full precision, pages of 32, a head size between the usual ones
        _attend("attend draft f32", "f32", ",".join(str(5 + (i * 1009 + 7) % 4096) for i in range(24)),
                ",".join(["5"] * 24), 16, 4, 80, 32),
        # pieces of prompts behind what the cache holds of them, beside single tokens
        _attend("attend prompts bf16", "bf16", "8192,4099,2048,777,300,1", "1024,1000,2048,1,1,1",
                32, 8, 128, 64),
        # one step of beam search, 8 sequences of 4 beams of which 2 go on: latency
        _fork("fork step", "17,130,500,1023,64,999,31,2000", 4, 2, 1, 8, 128, 16),
        # the same for 64 sequences of 8 beams over the 12 layers of a model
        _fork("fork layers", ",".join(str(33 + (i * 197 + 5) % 600) for i in range(64)), 8, 3, 12, 8, 128,
              32),
        # a small pool after some sequences have ended: latency
        _compact("compact small", 512, 301, 24, 1, 8, 64, 16),
        # a pool of twelve layers, 60 % in use
        _compact("compact layers", 2048, 1229, 64, 12, 8, 128, 32),
        # the pages of one sequence to another pool
        _copy("copy sequence", 1024, 65, 1, 8, 128, 16),
        # those of a whole batch, twelve layers
        _copy("copy layers", 1024, 601, 12, 8, 128, 32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(values):
    return ",".join(str(v) for v in values)


def draw(rng):
    op = rng.choice(["store", "store", "attend", "attend", "attend", "fork", "compact", "copy"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    dim = rng.choice([32, 64, 72, 80, 96, 128, 128])
    heads = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "store":
        count = _log_int(rng, 1, 64)
        total = _log_int(rng, count, max(count, 8000000 // (heads * dim * SIZE[dtype] // 2)))
        new = [rng.randint(0, 2 * total // count) for _ in range(count)]
        lens = [v + rng.choice([0, 0, rng.randint(0, 2000)]) for v in new]
        return _store(None, dtype, _text(lens), _text(new), heads, dim, page)
    if op == "attend":
        group = rng.choice([1, 2, 3, 4, 7, 8])
        q_heads = heads * group
        count = _log_int(rng, 1, 64)
        if rng.random() < 0.6:                        # decoding: one token or a few of each
            top = _log_int(rng, 1, max(1, min(16384, 150000000 // (count * heads * dim))))
            most = rng.choice([1, 1, 1, 2, 5, 8])
            lens = [rng.randint(1, top) for _ in range(count)]
            new = [min(most, v) for v in lens]
        else:                                         # pieces of prompts
            count = min(count, 8)
            top = _log_int(rng, 16, 8192 if dtype != "f32" else 2048)
            lens = [rng.randint(0, top) for _ in range(count)]
            new = [rng.choice([1, v, rng.randint(0, v)]) if v else 0 for v in lens]
        c = _attend(None, dtype, "", "", q_heads, heads, dim, page, rng.random() < 0.8)
        while True:
            c["lens"], c["new"] = _text(lens), _text(new)
            if work(c)["flops"] <= (1.3e11 if dtype != "f32" else 1.6e10):
                return c
            lens, new = [v * 3 // 4 for v in lens], [v * 3 // 4 for v in new]
    layers = rng.choice([1, 1, 2, 7, 12])
    bytes_of = _page_bytes(dict(dim=dim, heads=heads, page=page)) * layers
    most = max(16, min(4000, 400000000 // bytes_of))
    if op == "fork":
        beams = rng.choice([1, 2, 3, 4, 8])
        count = _log_int(rng, 1, max(1, min(64, most // (4 * beams))))
        room = max(1, (most // count - 2 * beams) * page // 2)
        lens = [rng.randint(0, min(room, 3000)) for _ in range(count)]
        return _fork(None, _text(lens), beams, rng.randint(1, beams), layers, heads, dim, page)
    pages = _log_int(rng, 4, most)
    if op == "compact":
        return _compact(None, pages, rng.randint(0, pages), rng.randint(1, 64), layers, heads, dim, page)
    return _copy(None, pages, rng.randint(1, pages), layers, heads, dim, page)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _randint(gen, high, shape):
    return torch.randint(0, high, shape, generator=gen, device="cuda")


def _shuffled(gen, n):
    return torch.randperm(n, generator=gen, device="cuda")


def _device(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _cu(lens):
    c = [0]
    for v in lens:
        c.append(c[-1] + v)
    return _device(c)


def _bytes(gen, shape):
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)


def _filled_pool(gen, pages, case):
    """A pool whose tokens hold rounded random keys and values, keys with some large channels."""
    h, d, page = case["heads"], case["dim"], case["page"]
    pool = torch.empty((pages, _page_bytes(case)), device="cuda", dtype=torch.uint8)
    wide = (torch.randn((h, d), generator=gen, device="cuda") * 0.5).exp()
    step = max(1, 100000000 // (page * h * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k, v = (_normal(gen, (n, page, h, d), torch.float32) for _ in range(2))
        pool[p:p + n] = _pack(*_encode(k * wide, case["dtype"]), *_encode(v, case["dtype"]))
    return pool


def _table(gen, lens, page, spare):
    """Rows of shuffled pages for sequences of these lengths: (table, pages of the pool)."""
    need = [-(-v // page) for v in lens]
    pages = sum(need) + spare
    order = _shuffled(gen, pages).to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def _counts(table, pages):
    held = table[table >= 0].long()
    return torch.bincount(held, minlength=pages).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    op, page = case["op"], case["page"]
    if op in ("store", "attend"):
        lens, new = _ints(case["lens"]), _ints(case["new"])
        table, pages = _table(gen, lens, page, 3)
        s.update(table=table, used=_device(lens), cu=_cu(new))
        dt, h, d = DTYPES[case["dtype"]], case["heads"], case["dim"]
        if op == "store":
            s["pool"] = _bytes(gen, (pages, _page_bytes(case)))
            # keys and values lie in the output of one projection, as slices of its rows
            kv = _normal(gen, (sum(new), 2 * h, d), torch.float32)
            kv[:, :h] *= (torch.randn((h, d), generator=gen, device="cuda") * 0.5).exp()
            kv = kv.to(dt)
            s["k"], s["v"] = kv[:, :h], kv[:, h:]
        else:
            s["pool"] = _filled_pool(gen, pages, case)
            s["q"] = _normal(gen, (sum(new), case["q_heads"], d), dt)
            for b, v in enumerate(lens):              # what nobody has written yet holds anything
                if v % page:
                    _spoil(s["pool"], int(table[b, v // page]), v % page, case)
    elif op == "fork":
        lens, beams, kept = _ints(case["lens"]), case["beams"], case["kept"]
        rows, width = [], max(-(-(v + 2) // page) for v in lens)
        at, used = 0, []
        for v in lens:                                # full pages shared, the last one each beam's own
            full, rest = v // page, v % page
            shared = list(range(at, at + full))
            at += full
            for _ in range(beams):
                rows.append(shared + ([at] if rest else []))
                at += 1 if rest else 0
                used.append(v)
        pages = at + 2 * len(rows) + 1
        order = _shuffled(gen, pages).to(torch.int32)
        table = torch.tensor([r + [-1] * (width - len(r)) for r in rows]).cuda()
        s["table"] = torch.where(table < 0, -1, order[table.clamp(min=0)]).to(torch.int32)
        s["used"] = _device(used)
        s["owners"] = _counts(s["table"], pages)
        # each sequence goes on from `kept` of its beams, each of them once at least
        parents = []
        for b in range(len(lens)):
            p = _shuffled(gen, beams)[:kept]
            more = p[_randint(gen, kept, (beams - kept,))]
            parents.append(b * beams + torch.cat((p, more))[_shuffled(gen, beams)])
        s["parents"] = torch.cat(parents).to(torch.int32)
        s["new"] = torch.ones(len(rows), dtype=torch.int32, device="cuda")
        s["pool"] = _bytes(gen, (case["layers"], pages, _page_bytes(case)))
    elif op == "compact":
        pages, live, rows = case["pages"], case["live"], case["rows"]
        held = _shuffled(gen, pages)[:live].to(torch.int32)
        width = max(1, -(-live // rows))
        flat = torch.full((rows * width,), -1, dtype=torch.int32, device="cuda")
        flat[:live] = held
        s["table"] = flat.view(rows, width)
        s["owners"] = _counts(s["table"], pages)
        s["pool"] = _bytes(gen, (case["layers"], pages, _page_bytes(case)))
    else:
        shape = (case["layers"], case["pages"], _page_bytes(case))
        s["pool"], s["other"] = _bytes(gen, shape), _bytes(gen, shape)
        s["src"], s["dst"] = (_shuffled(gen, case["pages"])[:case["count"]].to(torch.int32)
                              for _ in range(2))
    if own:
        from modulated_deformable_convolution_amd import attention, cache
        if op in ("store", "attend"):
            s["cache"] = cache.mdcn_cache_create(case["heads"], case["dim"], page)
        if op == "attend":
            s["handle"] = attention.mdcn_attention_create(case["q_heads"], case["heads"], case["dim"],
                                                          case["causal"])
    return s


def _spoil(pool, p, first, case):
    """Bytes of no meaning for the tokens of page p from `first` on."""
    n, h, strips = -(-case["dim"] // 32), case["heads"], case["page"] // 16
    strip = pool[p].view(h, strips, -1)
    for t in range(first, case["page"]):
        k = strip[:, t // 16]
        i = t % 16
        k[:, :256 * n].view(h, 4, 16, n * 4)[:, :, i] = 0x9e
        k[:, 256 * n:512 * n].view(h, 4, 16, n, 4)[:, i // 4, :, :, i % 4] = 0x57
        e = k[:, 512 * n:]
        w = 4 if n == 3 else n
        e[:, w * i:w * i + w] = 255
        e[:, 16 * w:].view(h, 4, n, 4)[:, i // 4, :, i % 4] = 255


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from modulated_deformable_convolution_amd import cache as C
    op = s["case"]["op"]
    if op == "store":
        C.store(s["cache"], s["pool"], s["k"], s["v"], s["table"], s["used"], s["cu"])
        k, v = C.load(s["cache"], s["pool"], s["table"], s["used"], s["cu"], s["k"].shape[0],
                      s["k"].dtype)
        return {"k": k, "v": v}
    if op == "attend":
        out, lse = C.attend(s["handle"], s["cache"], s["q"], s["pool"], s["table"], s["used"], s["cu"])
        return {"out": out, "lse": lse}
    if op == "fork":
        table, used, owners, short = C.fork_pages(s["pool"], s["table"], s["used"], s["owners"],
                                                  s["case"]["page"], s["parents"], s["new"])
        return {"pool": s["pool"], "table": table, "used": used, "owners": owners, "short": short}
    if op == "compact":
        table, owners, moved = C.compact_pages(s["pool"], s["table"], s["owners"])
        return {"pool": s["pool"], "table": table, "owners": owners, "moved": moved}
    C.copy_pages(s["pool"], s["other"], s["src"], s["dst"])
    return {"other": s["other"]}


# ------------------------------------------------------------------ the plain forms

def _encode(x, dtype):
    """[..., dim] fp32 -> (codes [..., blocks, 32], exponents [..., blocks]), both uint8."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))
    size = x.abs()
    m, e = torch.frexp(size.amax(-1))                 # m in [0.5, 1): at most 7 * 2^(e - 3) or (e - 2)
    lo, hi = EXPONENTS[dtype]
    e = torch.where(m == 0, lo, torch.where(m <= 0.875, e - 3, e - 2)).clamp(lo, hi)
    size = torch.ldexp(size, -e[..., None])
    code = torch.zeros_like(x, dtype=torch.uint8)
    for i, b in enumerate(BORDERS):
        code += (size >= b) if i % 2 else (size > b)
    return code | (x < 0).to(torch.uint8) << 3, (e + 127).to(torch.uint8)


def _pack(kc, ke, vc, ve):
    """[pages, page, heads, blocks(, 32)] -> [pages, page bytes]."""
    p, page, h, n = ke.shape
    kb, vb = (c[..., 0::2] | c[..., 1::2] << 4 for c in (kc, vc))
    s = page // 16
    k = kb.view(p, s, 16, h, n, 4, 4).permute(0, 3, 1, 5, 2, 4, 6).reshape(p, h, s, -1)
    v = vb.view(p, s, 4, 4, h, n, 16).permute(0, 4, 1, 2, 6, 5, 3).reshape(p, h, s, -1)
    if n == 3:
        ke = torch.nn.functional.pad(ke, (0, 1))
    kx = ke.view(p, s, 16, h, -1).permute(0, 3, 1, 2, 4).reshape(p, h, s, -1)
    vx = ve.view(p, s, 4, 4, h, n).permute(0, 4, 1, 2, 5, 3).reshape(p, h, s, -1)
    return torch.cat((k, v, kx, vx), -1).view(p, -1)


def _unpack(pages, case):
    """[pages, page bytes] -> (kc, ke, vc, ve) as _pack takes them."""
    h, n, s = case["heads"], -(-case["dim"] // 32), case["page"] // 16
    p, w = pages.shape[0], 4 if n == 3 else n
    k, v, kx, vx = pages.view(p, h, s, -1).split((256 * n, 256 * n, 16 * w, 16 * n), -1)
    k = k.reshape(p, h, s, 4, 16, n, 4).permute(0, 2, 4, 1, 5, 3, 6).reshape(p, 16 * s, h, n, 16)
    v = v.reshape(p, h, s, 4, 16, n, 4).permute(0, 2, 3, 6, 1, 5, 4).reshape(p, 16 * s, h, n, 16)
    kc, vc = (torch.stack((c & 15, c >> 4), -1).flatten(-2) for c in (k, v))
    ke = kx.reshape(p, h, s, 16, w).permute(0, 2, 3, 1, 4).reshape(p, 16 * s, h, w)[..., :n]
    ve = vx.reshape(p, h, s, 4, n, 4).permute(0, 2, 3, 5, 1, 4).reshape(p, 16 * s, h, n)
    return kc, ke, vc, ve


def _decode(code, e, dim):
    """fp32 values [..., dim] of codes and exponents."""
    size = torch.tensor(MAGNITUDES, device="cuda")[(code & 7).long()]
    x = torch.ldexp(torch.where(code > 7, -size, size), e.int()[..., None] - 127)
    return x.flatten(-2)[..., :dim]


def _fields(pool, case):
    """Views of a pool's bytes: keys [pages, heads, strips, g, token, blocks, 4], values
    [.., g, r, blocks, token], exponents [.., token, blocks] and [.., g, blocks, token]."""
    n = -(-case["dim"] // 32)
    w = 4 if n == 3 else n
    k, v, kx, vx = pool.view(pool.shape[0], case["heads"], case["page"] // 16, -1).split(
        (256 * n, 256 * n, 16 * w, 16 * n), -1)
    return (k.unflatten(-1, (4, 16, n, 4)), v.unflatten(-1, (4, 16, n, 4)),
            kx.unflatten(-1, (16, w))[..., :n], vx.unflatten(-1, (4, n, 4)))


def _plain_store(s):
    c, page = s["case"], s["case"]["page"]
    token = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu"].long(), token, right=True) - 1
    at = s["used"].long()[b] - s["cu"].long()[b + 1] + token
    p, strip, i = s["table"][b, at // page].long(), at % page // 16, at % 16
    kc, ke = _encode(s["k"].float(), c["dtype"])
    vc, ve = _encode(s["v"].float(), c["dtype"])
    kb, vb = (x[..., 0::2] | x[..., 1::2] << 4 for x in (kc, vc))        # [tokens, heads, n, 16]
    k, v, kx, vx = _fields(s["pool"], c)
    g, j = i // 4, i % 4
    k[p, :, strip, :, i] = kb.unflatten(-1, (4, 4)).transpose(2, 3)
    v[p, :, strip, g, :, :, j] = vb.transpose(2, 3)
    kx[p, :, strip, i] = ke
    vx[p, :, strip, g, :, j] = ve
    kb = k[p, :, strip, :, i].transpose(2, 3).flatten(-2)                # and read back
    vb = v[p, :, strip, g, :, :, j].transpose(2, 3)
    kc, vc = (torch.stack((x & 15, x >> 4), -1).flatten(-2) for x in (kb, vb))
    dt = s["k"].dtype
    return {"k": _decode(kc, kx[p, :, strip, i], c["dim"]).to(dt),
            "v": _decode(vc, vx[p, :, strip, g, :, j], c["dim"]).to(dt)}


def _plain_attend(s):
    c, q_all = s["case"], s["q"]
    page, d, h = c["page"], c["dim"], c["heads"]
    g = c["q_heads"] // h
    out = torch.zeros_like(q_all)
    lse = torch.full((c["q_heads"], q_all.shape[0]), -math.inf, device="cuda")
    at = 0
    for b, (length, n) in enumerate(zip(_ints(c["lens"]), _ints(c["new"]))):
        rows = slice(at, at + n)
        at += n
        if not n or not length:
            continue
        x = [x.flatten(0, 1)[:length] for x in
             _unpack(s["pool"][s["table"][b, :-(-length // page)].long()], c)]
        k = _decode(x[0], x[1], d).permute(1, 2, 0).contiguous()       # [heads, dim, keys]
        v = _decode(x[2], x[3], d).transpose(0, 1).contiguous()        # [heads, keys, dim]
        q = q_all[rows].float().view(n, h, g, d).permute(1, 2, 0, 3).reshape(h, g * n, d)
        scores = (q @ k * d ** -0.5).view(h, g, n, length)
        if c["causal"]:
            i, j = torch.arange(n, device="cuda"), torch.arange(length, device="cuda")
            scores = scores.masked_fill(j > i[:, None] + (length - n), -math.inf)
        top = scores.amax(-1, keepdim=True)
        e = (scores - top).exp()
        total = e.sum(-1, keepdim=True)
        o = ((e / total).view(h, g * n, length) @ v).view(h, g, n, d)
        out[rows] = o.permute(2, 0, 1, 3).reshape(n, h * g, d).to(out.dtype)
        lse[:, rows] = (top + total.log()).reshape(h * g, n)
    return {"out": out, "lse": lse}


def _plain_fork(s):
    page, pool, table = s["case"]["page"], s["pool"], s["table"]
    width = table.shape[1]
    parent = s["parents"].long()
    rows = torch.arange(parent.shape[0], device="cuda")
    first = torch.full((table.shape[0],), parent.shape[0], device="cuda").scatter_reduce(
        0, parent, rows, "amin")[parent] == rows
    used = s["used"].long()[parent]
    held, wants = -(-used // page), -(-(used + s["new"]) // page)
    j = torch.arange(width, device="cuda")
    old = table[parent]
    keep = j < held[:, None]
    copies = keep & (j == held[:, None] - 1) & ((used % page > 0) & ~first)[:, None]
    fresh = copies | ((j >= held[:, None]) & (j < wants[:, None]))
    result = torch.where(keep, old, -1)
    pages = s["owners"].shape[0]
    holds = s["owners"] - _counts(table, pages)
    shared = holds + _counts(torch.where(fresh, -1, result), pages)
    free = torch.nonzero(shared <= 0).flatten()
    at = torch.nonzero(fresh)
    result[at[:, 0], at[:, 1]] = free[:at.shape[0]].to(torch.int32)
    pool[:, result[copies].long()] = pool[:, old[copies].long()]
    return {"pool": pool, "table": result, "used": (used + s["new"]).to(torch.int32),
            "owners": holds + _counts(result, pages),
            "short": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _plain_compact(s):
    pool, table, owners = s["pool"], s["table"], s["owners"]
    live = owners > 0
    n = int(live.sum())
    number = torch.arange(owners.shape[0], device="cuda")
    src, dst = number[live & (number >= n)], number[~live & (number < n)]
    moved = torch.where(live, number, -1)
    moved[src] = dst
    pool[:, dst] = pool[:, src]
    counts = torch.zeros_like(owners)
    counts[moved[live]] = owners[live]
    rows = torch.where(table >= 0, moved[table.clamp(min=0).long()], -1)
    return {"pool": pool, "table": rows.to(torch.int32), "owners": counts,
            "moved": moved.to(torch.int32)}


def _plain_copy(s):
    s["other"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return {"other": s["other"]}


def run(state):
    if own:
        return _run_own(state)
    return {"store": _plain_store, "attend": _plain_attend, "fork": _plain_fork,
            "compact": _plain_compact, "copy": _plain_copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the cost

def _token_bytes(case):
    """Of one key or value head: 4 bits a channel, an exponent a block."""
    return -(-case["dim"] // 2) + -(-case["dim"] // 32)


def work(case):
    op = case["op"]
    if op == "store":
        values = sum(_ints(case["new"])) * case["heads"] * 2
        rounded = values * _token_bytes(case)
        return {"bytes": max(1, 2 * values * case["dim"] * SIZE[case["dtype"]] + 2 * rounded),
                "flops": 6 * values * case["dim"]}
    if op == "attend":
        lens, new, d = _ints(case["lens"]), _ints(case["new"]), case["dim"]
        pairs = sum(sum(max(0, v - n + 1 + i) for i in range(n)) if case["causal"] else n * v
                    for v, n in zip(lens, new))
        held = sum(v for v, n in zip(lens, new) if n)
        rows = sum(new) * case["q_heads"]
        return {"bytes": max(1, 2 * held * case["heads"] * _token_bytes(case) +
                             rows * (2 * d * SIZE[case["dtype"]] + 4)),
                "flops": 4 * d * case["q_heads"] * pairs}
    size = _page_bytes(case) * case["layers"]
    if op == "fork":
        lens, page, beams = _ints(case["lens"]), case["page"], case["beams"]
        copied = sum(1 for v in lens if v % page) * (beams - case["kept"])
        entries = sum(-(-v // page) for v in lens) * beams
        return {"bytes": 2 * copied * size + 8 * entries + 16 * len(lens) * beams, "flops": 0}
    if op == "compact":
        moves = case["live"] * (case["pages"] - case["live"]) // case["pages"]
        return {"bytes": 2 * moves * size + 8 * case["live"] + 12 * case["pages"], "flops": 0}
    return {"bytes": 2 * case["count"] * size + 8 * case["count"], "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_round(x, dtype):
    """Values that the cache holds for x [..., dim], one block at a time."""
    y = torch.empty_like(x, dtype=torch.float64)
    lo, hi = EXPONENTS[dtype]
    grid = torch.tensor([-v for v in MAGNITUDES[:0:-1]] + MAGNITUDES, device="cuda",
                        dtype=torch.float64)
    even = torch.tensor([i % 2 == 0 for i in range(7, 0, -1)] + [i % 2 == 0 for i in range(8)],
                        device="cuda")
    for c in range(0, x.shape[-1], 32):
        b = x[..., c:c + 32].double()
        top = b.abs().amax(-1, keepdim=True)
        e = torch.full_like(top, lo)
        for _ in range(hi - lo):
            e += (top > 7 * torch.pow(2.0, e)) & (e < hi)
        far = (b / torch.pow(2.0, e))[..., None] - grid
        # the nearest; of two that are as near, the one whose code is even
        best = (far.abs() * 4 - even.double() * 1e-12).argmin(-1)
        y[..., c:c + 32] = grid[best] * torch.pow(2.0, e)
    return y


def _token(pool, p, t, case):
    """Keys and values [heads, dim] in 64 bits of token t of each page of p, read by address."""
    n, h, d = -(-case["dim"] // 32), case["heads"], case["dim"]
    w, i = 4 if n == 3 else n, t % 16
    size = _strip_bytes(d)
    base = torch.arange(h, device="cuda")[:, None] * (case["page"] // 16) * size + t // 16 * size
    ch = torch.arange(d, device="cuda")[None]
    blk, c = ch // 32, ch % 32
    k_at = base + (((c // 8) * 16 + i) * n + blk) * 4 + c % 8 // 2
    v_at = base + 256 * n + (((i // 4) * 16 + c // 2) * n + blk) * 4 + i % 4
    ke_at = base + 512 * n + i * w + blk
    ve_at = base + 512 * n + 16 * w + ((i // 4) * n + blk) * 4 + i % 4
    sizes = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], device="cuda", dtype=torch.float64)
    r = []
    for at, e_at in ((k_at, ke_at), (v_at, ve_at)):
        byte = pool[p][:, at].long()
        code = torch.where(ch % 2 == 0, byte % 16, byte // 16)
        r.append(sizes[code] * torch.pow(2.0, pool[p][:, e_at].double() - 127))
    return r


def _exact_attend(s, case):
    d, page, h = case["dim"], case["page"], case["heads"]
    g = case["q_heads"] // h
    cu, lens = s["cu"].tolist(), s["used"].tolist()
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full((case["q_heads"], out.shape[0]), -math.inf, device="cuda", dtype=torch.float64)
    for b, length in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        n = cu[b + 1] - cu[b]
        if not n or not length:
            continue
        p = s["table"][b, :(length + page - 1) // page].long()
        tokens = [_token(s["pool"], p, t, case) for t in range(page)]
        k, v = (torch.stack([t[i] for t in tokens], 1).flatten(0, 1)[:length] for i in range(2))
        for head in range(case["q_heads"]):
            score = s["q"][rows, head].double() @ k[:, head // g].T / math.sqrt(d)
            if case["causal"]:
                hide = torch.ones((n, length), dtype=torch.bool, device="cuda")
                score[hide.triu(length - n + 1)] = -math.inf
            lse[head, rows] = torch.logsumexp(score, 1)
            out[rows, head] = (score - lse[head, rows][:, None]).exp() @ v[:, head // g]
    return {"out": out, "lse": lse}


def _exact_fork(s, case):
    page, table = case["page"], s["table"].tolist()
    used, owners = s["used"].tolist(), s["owners"].tolist()
    parents, new = s["parents"].tolist(), s["new"].tolist()
    width = len(table[0])
    for row in table:
        for p in row:
            if p >= 0:
                owners[p] -= 1
    result, todo, seen = [], [], set()
    for i, p in enumerate(parents):
        row, n = [-1] * width, used[p]
        for at in range(0, n, page):
            j = at // page
            if at + page > n and p in seen:
                todo.append((i, j, table[p][j]))
            else:
                row[j] = table[p][j]
                owners[row[j]] += 1
        todo += [(i, j, None) for j in range((n + page - 1) // page, (n + new[i] + page - 1) // page)]
        seen.add(p)
        result.append(row)
    free = [p for p, n in enumerate(owners) if n <= 0]
    for (i, j, source), p in zip(todo, free):
        result[i][j], owners[p] = p, 1
        if source is not None:
            s["pool"][:, p] = s["pool"][:, source]
    return {"pool": s["pool"], "table": _device(result),
            "used": _device([used[p] + n for p, n in zip(parents, new)]), "owners": _device(owners),
            "short": _device([0])}


def _exact_compact(s, case):
    owners, table = s["owners"].tolist(), s["table"].tolist()
    pages = len(owners)
    moved = [p if n > 0 else -1 for p, n in enumerate(owners)]
    count = sum(n > 0 for n in owners)
    holes = iter([p for p in range(count) if moved[p] < 0])
    for p in range(count, pages):
        if moved[p] >= 0:
            moved[p] = next(holes)
            s["pool"][:, moved[p]] = s["pool"][:, p]
    counts = [0] * pages
    for p, to in enumerate(moved):
        if to >= 0:
            counts[to] = owners[p]
    return {"pool": s["pool"], "table": _device([[moved[p] if p >= 0 else -1 for p in r] for r in table]),
            "owners": _device(counts), "moved": _device(moved)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "store":
        return {"k": _exact_round(s["k"], case["dtype"]), "v": _exact_round(s["v"], case["dtype"])}
    if op == "attend":
        return _exact_attend(s, case)
    if op == "fork":
        return _exact_fork(s, case)
    if op == "compact":
        return _exact_compact(s, case)
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        s["other"][:, b] = s["pool"][:, a]
    return {"other": s["other"]}
