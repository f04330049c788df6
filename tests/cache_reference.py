"""Plain forms of the 4-bit cache operators (CPU), straight from the definitions in
include/mdcn.h: one value, token or page at a time."""
import math

import torch

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LIMITS = {torch.float32: (-120, 125), torch.bfloat16: (-120, 125), torch.float16: (-23, 13)}
NAN_EXP = 255


# ---------------------------------------------------------------- rounding

def block_exponents(x, dtype):
    """[..., dim] -> [..., blocks]: the smallest e with max|x| <= 7 * 2^e, within the limits."""
    lo, hi = LIMITS[dtype]
    x = x.double()
    r = []
    for c in range(0, x.shape[-1], 32):
        top = x[..., c:c + 32].abs().amax(-1)
        e = torch.full(top.shape, hi, dtype=torch.int64)
        for v in range(hi - 1, lo - 1, -1):
            e[top <= 7 * 2.0 ** v] = v
        r.append(e)
    return torch.stack(r, -1)


def block_codes(x, e):
    """Codes [..., dim] of x at its blocks' exponents: nearest magnitude, ties to the even
    code, the sign in bit 3."""
    x = x.double()
    y = x.abs() / torch.repeat_interleave(2.0 ** e.double(), 32, -1)[..., :x.shape[-1]]
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64)
    y = y.clamp(max=6.0)
    far = (y[..., None] - grid).abs()
    near = far.amin(-1, keepdim=True)
    code = torch.full(y.shape, -1)
    for c in (1, 3, 5, 7, 0, 2, 4, 6):               # even codes last: they win ties
        code = torch.where(far[..., c] == near[..., 0], c, code)
    return code + 8 * (x < 0)


def rounded(x, dtype):
    """The values that a cache holds for x (no NaN among them), in 64 bits."""
    e = block_exponents(x, dtype)
    c = block_codes(x, e)
    m = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float64)[c]
    return m * torch.repeat_interleave(2.0 ** e.double(), 32, -1)[..., :x.shape[-1]]


def rounded_pair(k, v, dtype):
    """The same for keys and values with NaNs: both are NaN where either holds one."""
    bad = (k.isnan().any(-1) | v.isnan().any(-1))[..., None]
    r = []
    for x in (k, v):
        x = torch.where(bad, torch.zeros_like(x), x)
        r.append(torch.where(bad, math.nan, rounded(x, dtype)))
    return r


# ---------------------------------------------------------------- the layout

def strip_bytes(dim):
    n = -(-dim // 32)
    return 16 * (32 * n + (4 if n == 3 else n) + n)


def page_bytes(heads, dim, page):
    return heads * (page // 16) * strip_bytes(dim)


def value_places(dim, page, head, t, c):
    """Byte of the key's code, byte of the value's, bytes of their exponents, and the
    codes' shift within their bytes, of channel c of token t of a page."""
    n = -(-dim // 32)
    w = 4 if n == 3 else n
    base = (head * (page // 16) + t // 16) * strip_bytes(dim)
    i, b, ch = t % 16, c // 32, c % 32
    key = base + (((ch // 8) * 16 + i) * n + b) * 4 + (ch % 8) // 2
    value = base + 256 * n + (((i // 4) * 16 + ch // 2) * n + b) * 4 + i % 4
    key_e = base + 512 * n + i * w + b
    value_e = base + 512 * n + 16 * w + ((i // 4) * n + b) * 4 + i % 4
    return key, value, key_e, value_e, 4 * (ch % 2)


_places = {}


def _place_arrays(heads, dim, page):
    """value_places of every [page, heads, dim], as tensors."""
    at = _places.get((heads, dim, page))
    if at is None:
        at = torch.tensor([[[value_places(dim, page, h, t, c) for c in range(dim)]
                            for h in range(heads)] for t in range(page)]).unbind(-1)
        _places[(heads, dim, page)] = at
    return at


def write_token(pool, heads, dim, page, p, t, k, v, dtype):
    """Token t of page p from k, v [heads, dim]."""
    places = [x[t] for x in _place_arrays(heads, dim, page)]
    bad = k.isnan().any(-1) | v.isnan().any(-1)
    for which, x in enumerate((k, v)):
        x = torch.where(bad[:, None], torch.zeros_like(x), x)
        e = block_exponents(x, dtype)
        code = block_codes(x, e)
        e = e + 127
        if which == 0:
            e[bad] = NAN_EXP
        code = (code << places[4]).to(torch.uint8)
        at, at_e = places[which], places[2 + which]
        page_row = pool[p]
        page_row[at.flatten()] = 0                   # every byte belongs to two channels of x,
        for odd in range(2):                         # the last one's partner may be padding
            sel = (torch.arange(dim) % 2 == odd)
            page_row[at[:, sel].flatten()] |= code[:, sel].flatten()
        page_row[at_e.flatten()] = torch.repeat_interleave(e, 32, -1)[:, :dim].flatten().to(torch.uint8)


def read_page(pool, heads, dim, page, p):
    """Keys and values [page, heads, dim] of page p in 64 bits."""
    k_at, v_at, ke_at, ve_at, shift = _place_arrays(heads, dim, page)
    m = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float64)
    row = pool[p].long()
    nan = row[ke_at] == NAN_EXP
    return [torch.where(nan, math.nan, m[row[at] >> shift & 15] * 2.0 ** (row[e].double() - 127))
            for at, e in ((k_at, ke_at), (v_at, ve_at))]


def place(table, pages, page, b, at):
    """(page, token) of token `at` of row b, or None."""
    if at < 0 or at >= table.shape[1] * page:
        return None
    p = int(table[b, at // page])
    return (p, at % page) if 0 <= p < pages else None


def store(pool, heads, dim, page, k, v, table, used, cu, dtype):
    for b in range(len(used)):
        for t in range(cu[b], cu[b + 1]):
            at = place(table, pool.shape[0], page, b, used[b] - cu[b + 1] + t)
            if at:
                write_token(pool, heads, dim, page, *at, k[t], v[t], dtype)


def tokens(pool, heads, dim, page, table, b, places):
    """(keys, values [places, heads, dim], whether each has a page) of row b."""
    n = len(places)
    k, v = (torch.zeros(n, heads, dim, dtype=torch.float64) for _ in range(2))
    there = torch.zeros(n, dtype=torch.bool)
    pages = {}
    for i, at in enumerate(places):
        x = place(table, pool.shape[0], page, b, at)
        if x:
            if x[0] not in pages:
                pages[x[0]] = read_page(pool, heads, dim, page, x[0])
            k[i], v[i] = (y[x[1]] for y in pages[x[0]])
            there[i] = True
    return k, v, there


# ---------------------------------------------------------------- pages

def fork(pool, table, used, owners, page, parents, new):
    """(table, used, owners, missing), lists; pool [layers, pages, bytes] (or None) in place."""
    width = len(table[0]) if table else 0
    pages = len(owners)
    counts = list(owners)
    for row in table:
        for p in row:
            if 0 <= p < pages:
                counts[p] -= 1
    parents = list(range(len(table))) if parents is None else parents
    new = [0] * len(parents) if new is None else new
    result, lengths, needs, seen, excess = [], [], [], set(), 0
    for i, parent in enumerate(parents):
        row = [-1] * width
        held = 0
        n = 0
        if 0 <= parent < len(table):
            n = min(max(used[parent], 0), width * page)
            held = -(-n // page)
            for j in range(held):
                p = table[parent][j]
                if not 0 <= p < pages:
                    continue
                if j == held - 1 and n % page and parent in seen:
                    needs.append((i, j, p))
                else:
                    row[j] = p
                    counts[p] += 1
            seen.add(parent)
        more = max(new[i], 0)
        wants = -(-(n + more) // page)
        excess += max(0, wants - width)
        needs += [(i, j, None) for j in range(held, min(wants, width))]
        result.append(row)
        lengths.append(min(n + more, width * page))
    free = [p for p in range(pages) if counts[p] <= 0]
    missing = max(0, len(needs) - len(free)) + excess
    for (i, j, source), p in zip(needs, free):
        result[i][j] = p
        counts[p] = 1
        if source is not None and not missing and pool is not None:
            pool[:, p] = pool[:, source]
    return result, lengths, counts, missing


def compact(pool, table, owners):
    """(table, owners, moved), lists; pool in place."""
    pages = len(owners)
    held = [p for p in range(pages) if owners[p] > 0]
    n = len(held)
    moved = [-1] * pages
    holes = [p for p in range(n) if owners[p] <= 0]
    for p in held:
        moved[p] = p if p < n else holes.pop(0)
        if moved[p] != p:
            pool[:, moved[p]] = pool[:, p]
    counts = [0] * pages
    for p in held:
        counts[moved[p]] = owners[p]
    return ([[moved[p] if 0 <= p < pages else -1 for p in row] for row in table], counts, moved)
