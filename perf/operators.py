"""The operators of the 8-bit key/value cache, as cases to measure: writing, reading, attention.

The cache is paged: k_cache and v_cache hold e4m3 codes [pages, kv heads, slots of a page, D],
k_scale and v_scale one power of two (e8m0) for each page and head, and page_table [B, pages of a
sequence] says which page holds which positions.  Position p of sequence b is slot p % page of
page_table[b, p // page].

  write   new bf16 keys and values [B, H, L, D] go to positions starts[b] .. starts[b] + counts[b];
          a page's scale is the least power of two that keeps its largest magnitude within 448, and
          only grows while the page fills (codes already there are rescaled)
  read    positions starts[b] .. starts[b] + counts[b] come back as bf16 [B, H, L, D]
  attn    softmax attention of the last q_lens[b] tokens of each sequence over its kv_lens[b] cached
          ones: query heads share key/value heads in groups, causal by position, optionally within a
          window; bf16 O and the fp32 log-sum-exp of each row

`run` computes a case with plain torch operations, or (`own`) with the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one conversation, a short context: a step whose time is launch and latency
        attn("attn one short", B=1, Hq=32, Hkv=8, D=128, page=64, Lq=1, least=900, most=900),
        # a server's ordinary step: many conversations of all lengths, one token each
        attn("attn step ragged", B=48, Hq=32, Hkv=8, D=128, page=64, Lq=1, least=64, most=8192),
        # few conversations with very long contexts: the cache's bytes are all that counts
        attn("attn step long", B=2, Hq=32, Hkv=8, D=128, page=128, Lq=1, least=120001, most=131072),
        # checking drafted tokens: several queries a sequence, narrow heads, small pages
        attn("attn drafted", B=24, Hq=16, Hkv=2, D=64, page=16, Lq=5, least=100, most=4096, ragged=True),
        # every query head with its own cache head, the widest heads
        attn("attn own heads wide", B=4, Hq=8, Hkv=8, D=256, page=32, Lq=1, least=2000, most=3000),
        # a sliding-window layer's step over long contexts, the cache stored slot-major
        attn("attn step window", B=16, Hq=32, Hkv=8, D=128, page=64, Lq=1, least=1500, most=16384,
             window=1024, slot_major=True),
        # a long prompt taken in chunks: the last one, over everything before it
        attn("attn prompt chunk", B=1, Hq=32, Hkv=8, D=128, page=64, Lq=2048, least=16384, most=16384),
        # several prompts' next chunks together, each as long as it happens to be
        attn("attn chunks ragged", B=6, Hq=16, Hkv=4, D=64, page=16, Lq=509, least=600, most=5000, ragged=True),
        # the step's own keys and values, one token a sequence, into pages that are part full
        move("write", "write step", B=128, H=8, D=128, page=64, L=1, least=0, most=4000),
        # prompts that have just been computed
        move("write", "write prompts", B=8, H=8, D=128, page=64, L=8192, least=0, most=100, ragged=True),
        # a short prefix shared with a new request
        move("read", "read prefix", B=3, H=2, D=64, page=16, L=777, least=0, most=300),
        # whole contexts, to run the dense kernels on them
        move("read", "read contexts", B=4, H=16, D=128, page=64, L=16384, least=0, most=0),
    ]


def attn(name, B, Hq, Hkv, D, page, Lq, least, most, window=-1, ragged=False, slot_major=False):
    return dict(name=name, op="attn", B=B, Hq=Hq, Hkv=Hkv, D=D, page=page, Lq=Lq, least=least, most=most,
                window=window, ragged=ragged, slot_major=slot_major)


def move(op, name, B, H, D, page, L, least, most, ragged=False, slot_major=False):
    return dict(name=name, op=op, B=B, Hkv=H, D=D, page=page, L=L, least=least, most=most, ragged=ragged,
                slot_major=slot_major)


def draw(rng):
    def spread(lo, hi):   # whole numbers, even over the logarithm
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    H = rng.choice([1, 2, 4, 8, 8])
    slot_major = rng.random() < 0.3
    kind = rng.random()
    if kind < 0.15:
        L = spread(1, 8192)
        B = spread(1, max(1, min(128, 65536 * 1024 // (L * H * D))))
        c = move("write", "", B, H, D, page, L, 0, spread(16, 4000), rng.random() < 0.5, slot_major)
    elif kind < 0.3:
        L = spread(16, 16384)
        B = spread(1, max(1, min(64, 65536 * 1024 // (L * H * D))))
        c = move("read", "", B, H, D, page, L, 0, spread(16, 1000), rng.random() < 0.5, slot_major)
    else:
        G = rng.choice([1, 2, 4, 5, 8])
        Lq = 1 if kind < 0.6 else rng.randint(2, 9) if kind < 0.75 else spread(10, 2048)
        most = spread(max(Lq, 40), 131072 if Lq < 10 else 16384)
        room = 268435456 // (2 * H * D * most) if Lq < 10 else 150000000 // (Lq * most * H * G)
        B = spread(1, max(1, min(64, room)))
        if B * H * G * Lq * most * (4 * D) > 5.4e11:
            G, H = 1, min(H, 4)
        window = rng.choice([-1, -1, -1, spread(16, 4096)])
        c = attn("", B, H * G, H, D, page, Lq, max(Lq, most // rng.choice([1, 2, 20])), most, window,
                 rng.random() < 0.5, slot_major)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def evenly(lo, hi, n):
    """n whole numbers from lo to hi, hi among them."""
    return torch.tensor([hi - (hi - lo) * i // max(1, n - 1) for i in range(n)], dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    host = torch.Generator()
    host.manual_seed(int(seed))
    B, H, D, page, op = case["B"], case["Hkv"], case["D"], case["page"], case["op"]
    L = case["Lq"] if op == "attn" else case["L"]
    # lengths of the sequences: spaced evenly between the two bounds, in any order
    lens = evenly(case["least"], case["most"], B)[torch.randperm(B, generator=host)]
    new = torch.full((B,), L, dtype=torch.int32)
    if case["ragged"]:
        new = evenly((L + 1) // 2, L, B)[torch.randperm(B, generator=host)]
    ends = lens if op == "attn" else lens + L
    per_seq = -(-int(ends.max()) // page)
    # every sequence's pages lie anywhere in the pool, which has some to spare
    pages = -(-ends // page)
    pool = int(pages.sum()) + 3
    order = torch.randperm(pool, generator=host, dtype=torch.int32)
    table = torch.zeros(B, per_seq, dtype=torch.int32)
    mask = torch.arange(per_seq)[None, :] < pages[:, None]
    table[mask] = order[: int(pages.sum())]
    s = {"case": case, "table": table.to(DEV)}

    def cache():
        # what a model's keys and values look like: heads and pages of different strength, values
        # that fill the codes' range, and the page's power of two beside them
        shape = (pool, page, H, D) if case["slot_major"] else (pool, H, page, D)
        codes = torch.empty(shape, dtype=torch.uint8, device=DEV)
        step = max(1, 64 * 1024 * 1024 // (H * page * D))
        for at in range(0, pool, step):
            x = torch.randn((min(step, pool - at),) + shape[1:], generator=g, device=DEV)
            codes[at:at + step] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = codes.view(torch.float8_e4m3fn)
        if case["slot_major"]:
            codes = codes.permute(0, 2, 1, 3)
        scale = torch.randint(127 - 8, 127 - 5, (pool, H), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        return codes, scale.view(torch.float8_e8m0fnu)

    s["k_cache"], s["k_scale"] = cache()
    s["v_cache"], s["v_scale"] = cache()
    if op == "attn":
        s["q"] = torch.randn(B, case["Hq"], L, D, generator=g, device=DEV).to(torch.bfloat16)
        s["o"] = torch.zeros(B, case["Hq"], L, D, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.zeros(B, case["Hq"], L, device=DEV)
        s["kv_lens"] = lens.to(DEV)
        s["q_lens"] = new.to(DEV) if case["ragged"] else None
        s["window"] = None if case["window"] < 0 else case["window"]
    else:
        s["starts"] = lens.to(DEV)
        s["counts"] = new.to(DEV)
        if op == "write":
            # a projection's output [B, L, H, D], seen as [B, H, L, D]; a channel in 16 is stronger
            strong = 1 + 7 * (torch.arange(D, device=DEV) % 16 == 3)
            s["k"], s["v"] = ((torch.randn(B, L, H, D, generator=g, device=DEV) * strong).to(torch.bfloat16)
                              .permute(0, 2, 1, 3) for _ in range(2))
        else:
            s["k"], s["v"] = (torch.zeros(B, H, L, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    return s


# -------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        import io_aware_exact_fa2_gb300 as fa2
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"])
        if op == "write":
            fa2.fa2_cache_write(s["k"], s["v"], *cache, s["starts"], s["counts"])
            return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
        if op == "read":
            fa2.fa2_cache_read(*cache, s["k"], s["v"], s["starts"], s["counts"])
            return s["k"], s["v"]
        if "workspace" not in s:
            s["workspace"] = fa2.fa2_cache_attn_workspace(s["q"], s["k_cache"])
        fa2.fa2_cache_attn(s["q"], *cache, s["kv_lens"], s["o"], s["lse"], causal=True, q_lens=s["q_lens"],
                           window=s["window"], workspace=s["workspace"])
        return s["o"], s["lse"]
    if op == "write":
        for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
            plain_write(x, codes, scale, s["table"], s["starts"], s["counts"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "read":
        return tuple(plain_read(codes, scale, s["table"], s["starts"], s["counts"], x)
                     for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])))
    return plain_attn(s)


def power(e):
    """2.0 ** e in fp32 for whole -126 <= e <= 127, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def exponent(scale):
    """The exponent an e8m0 scale stands for."""
    return scale.view(torch.uint8).to(torch.int32) - 127


def plain_write(x, codes, scale, table, starts, counts):
    B, H, L, D = x.shape
    page = codes.shape[2]
    dev = x.device
    J = -(-L // page) + 1   # pages a sequence's new tokens can touch
    first = starts.long() // page
    col = first[:, None] + torch.arange(J, device=dev)
    token = col[:, :, None] * page + torch.arange(page, device=dev) - starts.long()[:, None, None]   # [B, J, page]
    fresh = (token >= 0) & (token < counts.long()[:, None, None])
    kept = (token < 0) & (col >= 0)[:, :, None]          # earlier tokens in the first page touched
    touched = fresh.any(2) & (col < table.shape[1])
    b = torch.arange(B, device=dev)[:, None, None]
    new = x.permute(0, 2, 1, 3)[b, token.clamp(0, L - 1)].float()                # [B, J, page, H, D]
    new = torch.where(fresh[..., None, None], new, 0.0)
    m, ex = torch.frexp(new.abs().amax(dim=(2, 4)))                                # [B, J, H]
    need = torch.where(m == 0, -96, ex - 9 + (m > 0.875).int()).clamp(-96, 119)
    ids = table.long().gather(1, col.clamp(max=table.shape[1] - 1))
    ids, touched = ids[touched], touched                                           # [n]
    need, new, fresh, kept = need[touched], new[touched], fresh[touched], kept[touched]
    old_e = exponent(scale)[ids]                                                  # [n, H]
    e = torch.where(kept.any(1)[:, None], torch.maximum(need, old_e), need)
    old = codes.view(torch.uint8)[ids]                                            # [n, H, page, D]
    moved = old.view(torch.float8_e4m3fn).float() * power((old_e - e).clamp(-126, 127))[:, :, None, None]
    new = (new.permute(0, 2, 1, 3) * power(-e)[:, :, None, None]).clamp(-448, 448)
    moved, new = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (moved, new))
    out = torch.where(fresh[:, None, :, None], new, torch.where(kept[:, None, :, None], moved, old))
    codes.view(torch.uint8)[ids] = out
    scale.view(torch.uint8)[ids] = (e + 127).to(torch.uint8)


def plain_gather(codes, scale, table):
    """All positions of each sequence in fp32: [B, H, positions, D]."""
    x = codes.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn).float()   # [B, M, H, page, D]
    x *= power(exponent(scale))[table.long()][..., None, None]
    B, M, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, M * page, D)


def plain_read(codes, scale, table, starts, counts, out):
    B, H, L, D = out.shape
    x = plain_gather(codes, scale, table)
    i = torch.arange(L, device=out.device)
    at = (starts.long()[:, None] + i).clamp(max=x.shape[2] - 1)
    x = x.gather(2, at[:, None, :, None].expand(B, H, L, D)).to(torch.bfloat16)
    return torch.where((i < counts[:, None])[:, None, :, None], x, out)


def plain_attn(s):
    q, kv_lens = s["q"], s["kv_lens"].long()
    B, Hq, L, D = q.shape
    k = plain_gather(s["k_cache"], s["k_scale"], s["table"])
    v = plain_gather(s["v_cache"], s["v_scale"], s["table"])
    H, n = k.shape[1], k.shape[2]
    i, j = torch.arange(L, device=q.device), torch.arange(n, device=q.device)
    q_lens = s["q_lens"].long() if s["q_lens"] is not None else torch.full_like(kv_lens, L)
    pos = (kv_lens - q_lens)[:, None] + i                                          # [B, L]
    seen = (j <= pos[:, :, None]) & (j < kv_lens[:, None, None])
    if s["window"] is not None:
        seen &= j >= pos[:, :, None] - s["window"]
    seen = seen[:, None, None]                                                     # [B, 1, 1, L, n]
    p = q.float().reshape(B, H, -1, D) @ k.transpose(2, 3)
    p = p.reshape(B, H, Hq // H, L, n).mul_(D ** -0.5).masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True).clamp(min=-3e38)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, -1, n) @ v).reshape(B, H, Hq // H, L, D) / total.clamp(min=1e-38)
    lse = (total.log() + top).reshape(B, Hq, L)
    o = o.reshape(B, Hq, L, D).to(torch.bfloat16)
    live = (i < q_lens[:, None])[:, None]                                          # rows past a sequence's own stay as they are
    return torch.where(live[..., None], o, s["o"]), torch.where(live, lse, s["lse"])


# ---------------------------------------------------------- work and exact values

def lengths(case):
    """Mean length of the sequences and of their new tokens."""
    B, L = case["B"], case["Lq"] if case["op"] == "attn" else case["L"]
    mean = float(evenly(case["least"], case["most"], B).double().mean())
    return mean, float(evenly((L + 1) // 2, L, B).double().mean()) if case["ragged"] else float(L)


def work(case):
    B, H, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    mean, new = lengths(case)
    if case["op"] != "attn":
        values = 2 * B * H * new * D
        return {"bytes": values * 3 + 2 * B * H * (new / page) + 8 * B, "flops": values}
    # keys that a sequence's queries see at all, and on average each
    keys, pairs = mean, mean - (new - 1) / 2
    if case["window"] >= 0:
        keys, pairs = min(keys, case["window"] + new), min(pairs, case["window"] + 1)
    rows = B * case["Hq"] * new
    return {"bytes": 2 * B * H * keys * (D + 1 / page) + 4 * B * keys / page + rows * (4 * D + 4),
            "flops": 4.0 * rows * pairs * D}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return exact_attn(case, s)
    return exact_write(case, s) if case["op"] == "write" else exact_read(case, s)


def two(e):
    """2.0 ** e in 64 bits for whole e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def values(codes, scale, ids):
    """The real numbers in the pages `ids` [n] of one cache, in 64 bits: [H, n * page, D]."""
    raw = codes[ids].contiguous().view(torch.uint8).to(torch.int64)
    sign, e, f = 1 - 2 * (raw >> 7), (raw >> 3) & 15, raw & 7
    x = sign * torch.where(e > 0, (8 + f) * two(e - 10), f * 2.0 ** -9)
    x = x * two(scale.view(torch.uint8)[ids].long() - 127)[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])


def exact_read(case, s):
    out = []
    for codes, scale, old in ((s["k_cache"], s["k_scale"], s["k"]), (s["v_cache"], s["v_scale"], s["v"])):
        y = old.double()
        for b in range(case["B"]):
            at, n = int(s["starts"][b]), int(s["counts"][b])
            x = values(codes, scale, s["table"][b].long())
            y[b, :, :n] = x[:, at:at + n]
        out.append(y)
    return tuple(out)


def exact_attn(case, s):
    B, Hq, H, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // H
    o, lse = s["o"].double(), s["lse"].double()
    for b in range(B):
        n = int(s["kv_lens"][b])
        m = case["Lq"] if s["q_lens"] is None else int(s["q_lens"][b])
        ids = s["table"][b, : -(-n // case["page"])].long()
        k, v = values(s["k_cache"], s["k_scale"], ids)[:, :n], values(s["v_cache"], s["v_scale"], ids)[:, :n]
        past = torch.arange(n, device=DEV)[None] - torch.arange(n - m, n, device=DEV)[:, None]   # key minus query
        hidden = past > 0
        if s["window"] is not None:
            hidden |= past < -s["window"]
        for h in range(Hq):
            w = (s["q"][b, h, :m].double() @ k[h // G].T) / math.sqrt(D)
            w[hidden] = -math.inf
            z = torch.logsumexp(w, 1)
            lse[b, h, :m] = z
            o[b, h, :m] = torch.exp(w - z[:, None]) @ v[h // G]
    return o, lse


def round_e4m3(x):
    """To the nearest e4m3 value, ties to an even fraction, in 64 bits."""
    step = two(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact_write(case, s):
    page, out = case["page"], []
    for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        y = codes.view(torch.uint8).view(torch.float8_e4m3fn).double()
        z = two(scale.view(torch.uint8).long() - 127)
        starts, counts, table = (s[n].tolist() for n in ("starts", "counts", "table"))
        if sum(counts) * case["Hkv"] * case["D"] > 2 ** 28:
            return None
        for b in range(case["B"]):
            at, end = starts[b], starts[b] + counts[b]
            while at < end:
                till = min(end, (at // page + 1) * page)
                p, slot = table[b][at // page], at % page
                rows = x[b, :, at - starts[b]:till - starts[b]].double()
                most = rows.abs().amax(dim=(1, 2))
                e = torch.floor(torch.log2(most.clamp(min=448 * 2.0 ** -96) / 448)).clamp(-96, 119) - 1
                for _ in range(2):   # the least exponent that holds `most`, whatever log2 rounded to
                    e = torch.where(most > 448 * two(e), (e + 1).clamp(max=119), e)
                new = two(e.clamp(min=-96))
                if slot:
                    new = torch.maximum(new, z[p])
                    y[p, :, :slot] = round_e4m3(y[p, :, :slot] * (z[p] / new)[:, None, None])
                y[p, :, slot:slot + till - at] = round_e4m3(rows / new[:, None, None])
                z[p] = new
                at = till
        out.append((y, z))
    return out[0][0], out[1][0], out[0][1], out[1][1]
