"""Timed cases of softmax attention beside the recurrences: the norm and
rotation of queries and keys, causal attention over packed or equal rows with
its gradients, the paged cache (plain or in 8 bits) and the attention of new
tokens over it.

``run`` computes a case in plain torch operations (32-bit, rounded once at the
end), or, with ``own`` set, by the library's calls.  ``exact`` gives the same
outputs from the definitions in 64 bits.

Query head h reads key head h // (Hq / Hk).  Over the tokens j <= i of a
sequence:
    s_ij = scale q_i . k_j,   y_i = sum_j exp(s_ij - lse_i) v_j
with lse_i = log sum_j exp(s_ij); a token with nothing to read has y = 0.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def _case(op, name, **kw):
    c = dict(op=op, name=name, **kw)
    if name is None:
        del c["name"]
    return c


def listed():
    return [
        # norm and rotation in a training step, q and k as views of one
        # projection's output, both directions
        _case("qk_norm", "qk_b8_t4096_h32_8_d64", B=8, T=4096, Hq=32, Hk=8, D=64, R=64, dtype="bf16",
              fused=True, train=True),
        # ... of one token for each of 256 users, half of each head rotated,
        # far positions: latency
        _case("qk_norm", "qk_b256_t1_h16_4_d128", B=256, T=1, Hq=16, Hk=4, D=128, R=64, dtype="bf16",
              fused=True, train=False),
        # prefill of a ragged set of prompts packed end to end (a serving step)
        _case("prompt", "prompt_packed24_t12288_h32_8_d128", B=1, T=12288, Hq=32, Hk=8, D=128, nseq=24,
              dtype="bf16", fused=True),
        # prefill of one long document
        _case("prompt", "prompt_b1_t16384_h32_4_d64", B=1, T=16384, Hq=32, Hk=4, D=64, nseq=0, dtype="bf16",
              fused=False),
        # a training step's attention and its gradients: small and odd, fp32
        _case("train", "train_b2_t300_h4_2_d64_f32", B=2, T=300, Hq=4, Hk=2, D=64, nseq=0, dtype="f32",
              fused=False),
        # ... at the size of a training batch, shared key heads, wide heads
        _case("train", "train_b4_t4096_h16_4_d128", B=4, T=4096, Hq=16, Hk=4, D=128, nseq=0, dtype="bf16",
              fused=False),
        # ... and the recurrence benchmark's training shape in bf16
        _case("train", "train_b8_t4096_h32_d64", B=8, T=4096, Hq=32, Hk=32, D=64, nseq=0, dtype="bf16",
              fused=False),
        # one token for each of 4 users at up to 2048 tokens: latency
        _case("decode", "decode_b4_len2048_h16_4_d128", B=4, T=1, Hq=16, Hk=4, D=128, len=2048, page=16,
              dtype="bf16", cache="same"),
        # one token for a full batch
        _case("decode", "decode_b64_len8192_h32_8_d128", B=64, T=1, Hq=32, Hk=8, D=128, len=8192, page=64,
              dtype="bf16", cache="same"),
        # four drafted tokens over two long documents, cache in 8 bits
        _case("decode", "decode_b2_t4_len131072_h32_8_d64_e4m3", B=2, T=4, Hq=32, Hk=8, D=64, len=131072,
              page=128, dtype="bf16", cache="e4m3"),
        # the keys and values of packed prompts into an 8-bit cache, and the
        # sequences back out of it (a prefix that is used again)
        _case("cache", "cache_packed24_t32768_h8_d128_e4m3", B=1, T=32768, Hk=8, D=128, nseq=24, len=0, page=64,
              dtype="bf16", cache="e4m3", read=True),
        # one token for each of 256 users into their pages: latency
        _case("cache", "cache_b256_t1_h4_d128", B=256, T=1, Hk=4, D=128, nseq=0, len=200, page=16,
              dtype="bf16", cache="same", read=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm", "prompt", "prompt", "train", "train", "decode", "decode", "cache"])
    dtype = rng.choice(["f32", "bf16", "bf16", "bf16"])
    D = rng.choice([64, 128])
    Hk = _log(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    fused = rng.random() < 0.4
    if op == "qk_norm":
        T = _log(rng, 1, 8192)
        B = _log(rng, 1, max(1, min(300, (1 << 17) // (T * Hk))))
        return _case(op, None, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D // 2, 32]), dtype=dtype,
                     fused=fused, train=rng.random() < 0.6)
    if op in ("prompt", "train"):
        # pairs of tokens times query heads, at most a fifth of the largest
        # listed case's of this kind; fp32 an eighth of that
        most = (1 << 29) // (8 if dtype == "f32" else 1)
        T = _log(rng, 1, min(8192, max(2, int(math.sqrt(most / Hq)))))
        B = _log(rng, 1, max(1, min(16, most // (Hq * T * T))))
        nseq = rng.choice([0, 0, _log(rng, 1, 40)])
        if nseq:
            T, B = min(B * T, int(math.sqrt(most / Hq))), 1
        return _case(op, None, B=B, T=T, Hq=Hq, Hk=Hk, D=D, nseq=nseq, dtype=dtype, fused=fused)
    cache = rng.choice(["same", "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "decode":
        B = _log(rng, 1, 200)
        return _case(op, None, B=B, T=rng.choice([1, 1, 1, 2, 5]), Hq=Hq, Hk=Hk, D=D,
                     len=_log(rng, 5, max(8, min(100000, (1 << 21) // (B * Hk)))), page=page, dtype=dtype, cache=cache)
    nseq = rng.choice([0, _log(rng, 1, 40)])
    T = _log(rng, 1, 20000 // Hk)
    B = 1 if nseq else _log(rng, 1, max(1, min(200, 20000 // (Hk * T))))
    return _case(op, None, B=B, T=T, Hk=Hk, D=D, nseq=nseq, len=_log(rng, 1, 400), page=page, dtype=dtype,
                 cache=cache, read=rng.random() < 0.7 or cache == "e4m3")


def _bytes(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    op, B, T, Hk, D, e = case["op"], case["B"], case["T"], case["Hk"], case["D"], _bytes(case["dtype"])
    if op == "cache":
        c = 1 + 4 / D if case["cache"] == "e4m3" else e
        n = 2.0 * B * T * Hk * D
        # k, v -> pages; pages -> k, v (the sequences' earlier tokens too)
        back = 2.0 * sum(_sizes(case, 0)[0]) * Hk * D if case["read"] else 0
        return {"bytes": n * (e + c) + back * (e + c), "flops": 4 * n + back}
    Hq = case["Hq"]
    if op == "qk_norm":
        n = float(B * T * (Hq + Hk) * D)
        return {"bytes": n * e * (5 if case["train"] else 2) + 4 * B * T, "flops": n * (30 if case["train"] else 10)}
    if op == "decode":
        c = 1 + 4 / D if case["cache"] == "e4m3" else e
        tokens = sum(_sizes(case, 0)[0])
        return {"bytes": 2.0 * tokens * Hk * D * c + 2.0 * B * T * Hq * D * e, "flops": 4.0 * tokens * T * Hq * D}
    lens = _sizes(case, 0)[0] if case["nseq"] else [T] * B
    pairs = sum(n * (n + 1) / 2 for n in lens) * Hq
    io = B * T * (2 * Hq + 2 * Hk) * D * e + B * T * Hq * 4
    if op == "prompt":
        return {"bytes": float(io), "flops": 4.0 * D * pairs}
    return {"bytes": float(2 * io + B * T * Hq * D * e), "flops": 14.0 * D * pairs}


# ----------------------------------------------------------------- the inputs

def _sizes(case, seed):
    """Lengths of a case's sequences, in all and of their new tokens.  Packed
    ones add up to T, an empty and a one-token sequence among them where there
    is room; in a decode batch one row may hold nothing (a padded batch)."""
    g = torch.Generator().manual_seed(seed * 2 + 1)
    n, T = case.get("nseq", 0), case["T"]
    if n:
        w = torch.rand(n, generator=g).add_(0.1)
        cuts = torch.floor(torch.cumsum(w, 0) / w.sum() * T).long()
        cuts[-1] = T
        if n > 3 and T > n:
            cuts[0], cuts[1] = 0, 1
        cuts = [0] + torch.cummax(cuts, 0).values.clamp_(max=T).tolist()
        new = [b - a for a, b in zip(cuts[:-1], cuts[1:])]
    else:
        new = [T] * case["B"]
    if case["op"] == "decode":
        at = torch.rand(case["B"], generator=g)
        have = [max(T, int(case["len"] * (0.5 + 0.5 * x))) for x in at.tolist()]
        if case["B"] > 4:
            have[2] = 0
        return have, new
    if case["op"] == "cache":
        # earlier tokens: the same number in all for every seed
        return [m + int(case["len"] * (0.618 * i % 1)) for i, m in enumerate(new)], new
    return new, new


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt, op = DTYPES[case["dtype"]], case["op"]
    B, T, Hk, D = (case[n] for n in ("B", "T", "Hk", "D"))

    def rn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    st = {"case": case}
    have, new = _sizes(case, int(seed))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st.update(have=have, starts=starts, seq_starts=None)
    if case.get("nseq"):
        st["seq_starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if op in ("qk_norm", "prompt", "train"):
        Hq = case["Hq"]
        if case["fused"]:   # the projection's output, [queries | keys | values]
            qkv = rn(B, T, Hq + 2 * Hk, D).to(dt)
            st.update(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hk], v=qkv[:, :, Hq + Hk:])
        else:
            st.update(q=rn(B, T, Hq, D).to(dt), k=rn(B, T, Hk, D).to(dt), v=rn(B, T, Hk, D).to(dt))
    if op == "qk_norm":
        R = case["R"]
        st.update(wq=1 + 0.1 * rn(D), wk=1 + 0.1 * rn(D),
                  theta=10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float32) / R))
        # each row at a place of its own in a sequence
        first = torch.randint(0, 100000 if T == 1 else 1000, (B, 1), generator=gen, device=dev)
        st["positions"] = (first + torch.arange(T, device=dev)).to(torch.int32)
        if case["train"]:
            st.update(dq=rn(B, T, Hq, D).to(dt), dk=rn(B, T, Hk, D).to(dt))
        return st
    if op in ("prompt", "train"):
        st["plan"] = _pad_plan(starts, dev) if case["nseq"] else None
        if op == "train":
            st["dy"] = rn(B, T, Hq, D).to(dt)
        return st

    # the cache: pages in no order, some of them nobody's
    page = case["page"]
    most = max(1, max((n + page - 1) // page for n in have))
    pages = len(have) * most + 3
    st["table"] = torch.randperm(pages, generator=gen, device=dev)[:len(have) * most].view(-1, most).to(torch.int32)
    st["lens"] = torch.tensor(have, dtype=torch.int32, device=dev)
    kc = (rn(pages, Hk, page, D).to(dt), rn(pages, Hk, page, D).to(dt))
    if case["cache"] == "e4m3":
        packed = [_quantise(x.float()) for x in kc]
        st.update(k_pages=packed[0][0], v_pages=packed[1][0], k_scale=packed[0][1], v_scale=packed[1][1])
    else:
        st.update(k_pages=kc[0], v_pages=kc[1], k_scale=None, v_scale=None)
    if op == "decode":
        st["q"] = rn(B, T, case["Hq"], D).to(dt)
    else:
        st.update(k=rn(B, T, Hk, D).to(dt), v=rn(B, T, Hk, D).to(dt))
        st["out_starts"], st["total"] = None, sum(have)
        if case["read"]:
            cuts = [0]
            for n in have:
                cuts.append(cuts[-1] + n)
            st["out_starts"] = torch.tensor(cuts, dtype=torch.int32, device=dev)
    return st


def _pad_plan(starts, dev):
    """Where each sequence's tokens go in a padded batch, and back."""
    begin = torch.tensor(starts[:-1], device=dev)[:, None]
    size = torch.tensor(starts[1:], device=dev)[:, None] - begin
    at = torch.arange(max(1, int(size.max())), device=dev)[None]
    inside = at < size
    return {"take": torch.where(inside, begin + at, 0), "inside": inside}


def _quantise(x):
    """fp32 [..., D] as e4m3 values and their scale: the largest magnitude of
    the D entries stands for the type's largest value."""
    scale = x.abs().amax(-1) / E4M3_MAX
    safe = torch.where(scale > 0, scale, 1.0)
    return (x / safe[..., None]).to(torch.float8_e4m3fn), scale


# ------------------------------------------------------------ the plain forms

def _turns(st):
    """cos and sin of every token's angles, [B, T, 1, R / 2]."""
    angle = st["positions"].double()[..., None] * st["theta"].double()
    return torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]


def _norm_turn(x, w, cos, sin, R):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1)


def _norm_turn_back(dz, x, w, cos, sin, R):
    a, b = dz[..., :R // 2].float(), dz[..., R // 2:R].float()
    dz = torch.cat((a * cos + b * sin, b * cos - a * sin, dz[..., R:].float()), -1)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn = x * r
    dn = dz * w
    return r * (dn - xn * (dn * xn).mean(-1, keepdim=True)), (dz * xn).sum((0, 1, 2))


def _plain_qk_norm(st):
    dt, R = st["q"].dtype, st["case"]["R"]
    cos, sin = _turns(st)
    out = {"q": _norm_turn(st["q"], st["wq"], cos, sin, R).to(dt), "k": _norm_turn(st["k"], st["wk"], cos, sin, R).to(dt)}
    if st["case"]["train"]:
        dq, out["dwq"] = _norm_turn_back(st["dq"], st["q"], st["wq"], cos, sin, R)
        dk, out["dwk"] = _norm_turn_back(st["dk"], st["k"], st["wk"], cos, sin, R)
        out.update(dq=dq.to(dt), dk=dk.to(dt))
    return out


def _plain_attention(st, backward):
    """Rows of queries in blocks, each against the keys up to its end."""
    case, dt, plan = st["case"], st["q"].dtype, st["plan"]
    Hq, Hk, D = (case[n] for n in ("Hq", "Hk", "D"))
    group, scale = Hq // Hk, D ** -0.5

    def lay(x, heads):   # [B * heads, T, D] fp32, packed sequences as a padded batch
        x = x.float()
        if plan is not None:
            x = x[0][plan["take"]] * plan["inside"][:, :, None, None]
        return x.transpose(1, 2).reshape(x.shape[0] * heads, x.shape[1], D)

    def unlay(x, heads):
        x = x.view(-1, heads, x.shape[1], D).transpose(1, 2)
        return (x if plan is None else x[plan["inside"]][None]).to(dt).contiguous()

    q, k, v = lay(st["q"], Hq), lay(st["k"], Hk), lay(st["v"], Hk)
    n, T = k.shape[:2]
    q = q.view(n, group, T, D)
    kt, vt = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    y, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
    if backward:
        dy, dq = lay(st["dy"], Hq).view(n, group, T, D), torch.empty_like(q)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    block = max(1, min(T, (1 << 30) // (n * group * T)))
    for lo in range(0, T, block):
        hi = min(T, lo + block)
        rows = torch.arange(lo, hi, device=q.device).repeat(group)
        hidden = rows[:, None] < torch.arange(hi, device=q.device)
        qb = q[:, :, lo:hi].reshape(n, -1, D)
        s = torch.bmm(qb, kt[:, :, :hi].contiguous()).mul_(scale).masked_fill_(hidden, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        lse[:, :, lo:hi] = (m + torch.log(total)).view(n, group, -1)
        p = p.div_(total)
        yb = torch.bmm(p, v[:, :hi])
        y[:, :, lo:hi] = yb.view(n, group, -1, D)
        if backward:
            db = dy[:, :, lo:hi].reshape(n, -1, D)
            dv[:, :hi] += torch.bmm(p.transpose(1, 2), db)
            ds = torch.bmm(db, vt[:, :, :hi].contiguous()).sub_((db * yb).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            dq[:, :, lo:hi] = torch.bmm(ds, k[:, :hi]).view(n, group, -1, D)
            dk[:, :hi] += torch.bmm(ds.transpose(1, 2), qb)
    lse = lse.view(-1, Hq, T).transpose(1, 2)
    lse = (lse if plan is None else lse[plan["inside"]][None]).contiguous()
    out = {"y": unlay(y.view(-1, T, D), Hq), "lse": lse}
    if backward:
        out.update(dq=unlay(dq.view(-1, T, D), Hq), dk=unlay(dk, Hk), dv=unlay(dv, Hk))
    return out


def _dense(st, pages, scale):
    """The rows' pages as [B, Hk, most * page, D] fp32."""
    x = pages[st["table"].long()] if scale is None else pages.view(torch.uint8)[st["table"].long()].view(pages.dtype)
    x = x.float()
    if scale is not None:
        x = x * scale[st["table"].long()][..., None]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _plain_decode(st):
    case = st["case"]
    B, T, Hq, Hk, D = (case[n] for n in ("B", "T", "Hq", "Hk", "D"))
    group = Hq // Hk
    k, v = _dense(st, st["k_pages"], st["k_scale"]), _dense(st, st["v_pages"], st["v_scale"])
    L = k.shape[2]
    q = st["q"].float().view(B, T, Hk, group, D).permute(0, 2, 1, 3, 4).reshape(B * Hk, T * group, D)
    s = torch.bmm(q, k.view(B * Hk, L, D).transpose(1, 2).contiguous()) * D ** -0.5
    # token t of a row sees all but the T - 1 - t last tokens
    sees = st["lens"][:, None] - (T - 1) + torch.arange(T, device=s.device)
    seen = (torch.arange(L, device=s.device) < sees[..., None])[:, None, :, None]
    s = s.view(B, Hk, T, group, L).masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    y = torch.bmm(p.view(B * Hk, T * group, L), v.view(B * Hk, L, D)).view(B, Hk, T, group, D)
    y = y / torch.where(total > 0, total, 1.0)
    return {"y": y.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(st["q"].dtype)}


def _places(starts, have, dev):
    """Row and position of every token of sequences that end at `have`."""
    size = torch.tensor(starts[1:], device=dev) - torch.tensor(starts[:-1], device=dev)
    row = torch.repeat_interleave(torch.arange(len(have), device=dev), size)
    at = torch.arange(starts[-1], device=dev) - torch.tensor(starts, device=dev)[row]
    return row, at + (torch.tensor(have, device=dev) - size)[row]


def _plain_cache(st):
    case, dev = st["case"], st["k"].device
    Hk, D, page = (case[n] for n in ("Hk", "D", "page"))
    row, at = _places(st["starts"], st["have"], dev)
    p, o = st["table"].long()[row, at // page], at % page
    for name in ("k", "v"):
        x, pages, scale = st[name].reshape(-1, Hk, D), st[name + "_pages"], st[name + "_scale"]
        if scale is None:
            pages[p, :, o] = x
        else:
            x, s = _quantise(x.float())
            pages.view(torch.uint8)[p, :, o] = x.view(torch.uint8)
            scale[p, :, o] = s
    if not case["read"]:
        return {"k": st["k_pages"], "v": st["v_pages"]}
    cuts = [0]
    for n in st["have"]:
        cuts.append(cuts[-1] + n)
    row, at = _places(cuts, st["have"], dev)
    p, o, out = st["table"].long()[row, at // page], at % page, {}
    for name in ("k", "v"):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        if scale is None:
            out[name] = pages[p, :, o][None]
        else:
            x = pages.view(torch.uint8)[p, :, o].view(pages.dtype).float() * scale[p, :, o][..., None]
            out[name] = x.to(st["k"].dtype)[None]
    return out


# --------------------------------------------------------- the library's calls

def _own_qk_norm(st):
    from linear_attention_rnn_wkv7_amd import api

    args = [st[n] for n in ("q", "k", "wq", "wk", "theta", "positions")]
    q, k = api.qk_norm_forward(*args, eps=EPS)
    out = {"q": q, "k": k}
    if st["case"]["train"]:
        out.update(api.qk_norm_backward(st["dq"], st["dk"], *args, eps=EPS))
    return out


def _own_attention(st, backward):
    from linear_attention_rnn_wkv7_amd import api

    args = [st[n] for n in ("q", "k", "v")]
    y, lse, rec = api.attn_forward(*args, seq_starts=st["seq_starts"], want_lse=True, want_record=backward)
    out = {"y": y, "lse": lse}
    if backward:
        out.update(api.attn_backward(*args, y, lse, st["dy"], rec, seq_starts=st["seq_starts"]))
    return out


def _own_decode(st):
    from linear_attention_rnn_wkv7_amd import api

    return {"y": api.attn_decode(*(st[n] for n in ("q", "k_pages", "v_pages", "table", "lens", "k_scale", "v_scale")))}


def _own_cache(st):
    from linear_attention_rnn_wkv7_amd import api

    cache = [st[n] for n in ("k_pages", "v_pages", "table", "lens", "k_scale", "v_scale")]
    api.kv_write(st["k"], st["v"], *cache, seq_starts=st["seq_starts"])
    if not st["case"]["read"]:
        return {"k": st["k_pages"], "v": st["v_pages"]}
    k, v = api.kv_read(*cache, T=st["total"], seq_starts=st["out_starts"], dtype=st["k"].dtype)
    return {"k": k, "v": v}


def run(state):
    op = state["case"]["op"]
    if op == "qk_norm":
        return _own_qk_norm(state) if own else _plain_qk_norm(state)
    if op == "decode":
        return _own_decode(state) if own else _plain_decode(state)
    if op == "cache":
        return _own_cache(state) if own else _plain_cache(state)
    return _own_attention(state, op == "train") if own else _plain_attention(state, op == "train")


# ------------------------------------------------------- the definition, 64 bits

def _exact_qk_norm(st):
    case, R = st["case"], st["case"]["R"]
    # a rotation is the product with a unit complex number
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=st["q"].device),
                       st["positions"].double()[:, :, None, None] * st["theta"].double())
    out = {}
    for n in ("q", "k"):
        x = st[n].double().requires_grad_()
        w = st["w" + n].double().requires_grad_()
        h = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + EPS) * w
        z = torch.complex(h[..., :R // 2], h[..., R // 2:R]) * unit
        z = torch.cat((z.real, z.imag, h[..., R:]), -1)
        out[n] = z.detach()
        if case["train"]:
            out["d" + n], out["dw" + n] = torch.autograd.grad(z, (x, w), st["d" + n].double())
    return out


def _exact_attention(st, backward):
    """One sequence and query head at a time, some rows of it at once."""
    case = st["case"]
    Hq, Hk, D = (case[n] for n in ("Hq", "Hk", "D"))
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    B, T = q.shape[:2]
    y, lse = torch.zeros_like(q), torch.zeros_like(q[..., 0])
    if backward:
        dy = st["dy"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    starts = st["starts"]
    seqs = [(0, a, b) for a, b in zip(starts[:-1], starts[1:])] if case["nseq"] else [(b, 0, T) for b in range(B)]
    for b, lo, hi in seqs:
        for h in range(Hq):
            g = h * Hk // Hq
            K, V = k[b, lo:hi, g], v[b, lo:hi, g]
            for at in range(lo, hi, 4096):
                to = min(hi, at + 4096)
                Kn, Vn = K[:to - lo], V[:to - lo]
                z = q[b, at:to, h] @ Kn.T / math.sqrt(D)
                z += torch.full_like(z, -math.inf).triu(at - lo + 1)
                lse[b, at:to, h] = torch.logsumexp(z, -1)
                P = torch.softmax(z, -1)
                y[b, at:to, h] = P @ Vn
                if not backward:
                    continue
                G = dy[b, at:to, h]
                dv[b, lo:to, g] += P.T @ G
                dP = G @ Vn.T
                dz = P * (dP - (P * dP).sum(-1, keepdim=True)) / math.sqrt(D)
                dq[b, at:to, h] = dz @ Kn
                dk[b, lo:to, g] += dz.T @ q[b, at:to, h]
    out = {"y": y, "lse": lse}
    if backward:
        out.update(dq=dq, dk=dk, dv=dv)
    return out


def _exact_rows(st, row):
    """The cached tokens of a row in order: k and v [tokens, Hk, D]."""
    case, n = st["case"], st["have"][row]
    out = []
    for name in ("k", "v"):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        mine = st["table"][row].tolist()
        x = torch.stack([pages[p].double() * (1 if scale is None else scale[p].double()[..., None]) for p in mine])
        out.append(x.transpose(1, 2).reshape(-1, case["Hk"], case["D"])[:n])
    return out


def _exact_decode(st):
    case, q = st["case"], st["q"].double()
    B, T, Hq, Hk, D = (case[n] for n in ("B", "T", "Hq", "Hk", "D"))
    y = torch.zeros_like(q)
    for b in range(B):
        k, v = _exact_rows(st, b)
        for t in range(T):
            n = st["have"][b] - (T - 1 - t)
            if n <= 0:
                continue
            for g in range(Hk):
                mine = slice(g * (Hq // Hk), (g + 1) * (Hq // Hk))
                P = torch.softmax(q[b, t, mine] @ k[:n, g].T / math.sqrt(D), -1)
                y[b, t, mine] = P @ v[:n, g]
    return {"y": y}


def _nearest_e4m3(x):
    """The e4m3 value nearest to x (fp64, at most 448 in magnitude), ties to
    the even one."""
    size = x.abs()
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.where(size > 0, size, 1.0))), min=-6) - 3)
    return torch.sign(x) * torch.round(size / step) * step


def _exact_cache(st):
    case = st["case"]
    page, dt, out = case["page"], st["k"].dtype, {}
    if not case["read"]:   # copies: the same values at the same places
        for name in ("k", "v"):
            x, pages = st[name].flatten(0, 1), st[name + "_pages"].double()
            for s, n in enumerate(st["have"]):
                m = st["starts"][s + 1] - st["starts"][s]
                for j in range(m):
                    at = n - m + j
                    pages[st["table"][s, at // page], :, at % page] = x[st["starts"][s] + j].double()
            out[name] = pages
        return out
    for name in ("k", "v"):
        x, parts = st[name].flatten(0, 1), []
        for s, n in enumerate(st["have"]):
            old = _exact_rows(st, s)[name == "v"]
            m = st["starts"][s + 1] - st["starts"][s]
            new = x[st["starts"][s]:st["starts"][s + 1]].double()
            if case["cache"] == "e4m3":
                # the scale is an fp32 number by definition, and so is the quotient
                scale = new.float().abs().amax(-1, keepdim=True) / E4M3_MAX if m else new.float()[..., :1]
                ratio = (new.float() / torch.where(scale > 0, scale, 1.0)).double()
                new = _nearest_e4m3(ratio) * scale.double()
            parts.append(torch.cat((old[:n - m], new)))
        out[name] = torch.cat(parts)[None]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "qk_norm":
        return _exact_qk_norm(st)
    if case["op"] == "decode":
        return _exact_decode(st)
    if case["op"] == "cache":
        return _exact_cache(st)
    return _exact_attention(st, case["op"] == "train")
