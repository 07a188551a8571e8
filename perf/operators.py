"""The attention operators next to the indexer, case by case: what a serving program calls before and after a
layer's selection.

norm_rope  li_norm_rope: RMS norms of query and key heads, with the rotation of their rotary part
append     li_append_paged: latent rows normed, rotated and written into a paged cache
latent     li_latent_attention: absorbed queries over the paged latent, the selected positions or the whole prefix
prompt     li_prompt_attention: expanded keys and values of whole prompts, causal, ragged batches

`own` False computes the plain form in elementary torch operations; True makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 10000.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token of four sequences: 64 query heads of 128 and the one indexer key, half of each rotated
        dict(name="norm_rope_decode", op="norm_rope", n=4, hq=64, hk=1, dim=128, rope=64, halves=False, dtype="bf16", far=131072),
        # a prompt's queries and rotary keys at the width of attention heads (128 + 64)
        dict(name="norm_rope_prompt", op="norm_rope", n=8192, hq=64, hk=1, dim=192, rope=64, halves=True, dtype="bf16", far=65536),
        # one decode token for each of eight sequences into a shuffled page pool
        dict(name="append_decode", op="append", batch=8, T=1, d_v=512, rope=64, page=64, lo=1000, hi=4000, dtype="bf16"),
        # prompts of uneven length, written in one call
        dict(name="append_prompt", op="append", batch=4, T=8192, d_v=512, rope=64, page=64, lo=0, hi=1000, dtype="bf16"),
        # the attention after one decode token's selection: 2048 of 8192 positions
        dict(name="select_decode", op="latent", batch=1, T=1, H=64, d_v=512, rope=64, page=64, lo=8192, hi=8192, k=2048, dtype="bf16"),
        # a decode batch with ragged prefixes of 16K to 32K, 128 heads
        dict(name="select_batch", op="latent", batch=8, T=1, H=128, d_v=512, rope=64, page=64, lo=16384, hi=32768, k=2048, dtype="bf16"),
        # part of a prefill chunk at the end of a 64K prefix: each query with its own 2048 positions
        dict(name="select_chunk", op="latent", batch=1, T=256, H=32, d_v=512, rope=64, page=64, lo=65536, hi=65536, k=2048, dtype="bf16"),
        # no selection: the whole prefix at 128K, the layers that a model keeps dense
        dict(name="dense_long", op="latent", batch=4, T=1, H=64, d_v=512, rope=64, page=64, lo=131072, hi=131072, k=0, dtype="bf16"),
        # the smallest configuration's latent in fp32, odd page size
        dict(name="dense_f32", op="latent", batch=2, T=1, H=8, d_v=32, rope=16, page=17, lo=300, hi=512, k=0, dtype="f32"),
        # short prompts of a mixed batch, where every position is selected
        dict(name="prompt_short", op="prompt", batch=8, lo=1, hi=257, past=0, H=16, nope=128, rope=64, d_v=128, dtype="bf16"),
        # four prompts of up to 2048 positions, the longest that need no selection
        dict(name="prompt_2k", op="prompt", batch=4, lo=1500, hi=2048, past=0, H=32, nope=128, rope=64, d_v=128, dtype="bf16"),
        # one long prompt
        dict(name="prompt_8k", op="prompt", batch=1, lo=8192, hi=8192, past=0, H=32, nope=128, rope=64, d_v=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "latent", "latent", "prompt"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if op == "norm_rope":
        dim = rng.choice([64, 96, 128, 192, 256])
        rope = rng.choice([r for r in (0, 32, 64, 128) if r <= dim])
        return dict(op=op, n=_log(rng, 1, 4096), hq=rng.randint(1, 64), hk=rng.randint(0, 4), dim=dim, rope=rope,
                    halves=rng.random() < 0.5, dtype=dtype, far=_log(rng, 16, 1 << 20))
    d_v, rope = rng.choice([(512, 64), (512, 64), (256, 64), (128, 64), (192, 0), (64, 32), (32, 16)])
    if op == "append":
        return dict(op=op, batch=rng.randint(1, 16), T=_log(rng, 1, 2000), d_v=d_v, rope=rope,
                    page=rng.choice([1, 16, 17, 64, 128]), lo=0, hi=_log(rng, 10, 4000), dtype=dtype)
    if op == "latent":
        hi = _log(rng, 1, 4096 if dtype == "f32" else 65536)
        T = rng.choice([1, 1, 1, 2, 3, 7])
        k = rng.choice([0, 1]) * _log(rng, 1, 2048)
        return dict(op=op, batch=rng.randint(1, 6), T=T, H=rng.choice([1, 8, 16, 20, 32, 64, 128]), d_v=d_v, rope=rope,
                    page=rng.choice([1, 16, 17, 64, 128]), lo=rng.randint(0, hi), hi=hi, k=k, dtype=dtype)
    hi = _log(rng, 1, 256 if dtype == "f32" else 4096)
    return dict(op=op, batch=rng.randint(1, 4), lo=rng.randint(0, hi), hi=hi, past=rng.choice([0, 0, rng.randint(1, 1000)]),
                H=rng.choice([1, 4, 8, 16]), nope=rng.choice([64, 128]), rope=rng.choice([0, 32, 64]),
                d_v=rng.choice([64, 128]), dtype=dtype)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], both ends among them, in a mixed order."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 5 + 3) % n if n % 5 else i) // (n - 1) for i in range(n)]


def _lengths(case):
    """Positions already there, one number a sequence."""
    return _spread(case["lo"], case["hi"], case["batch"])


def _new(case):
    """append: rows that each sequence gets, the last one all of T."""
    return _spread((case["T"] + 1) // 2, case["T"], case["batch"])


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _inv_freq(rope):
    return (THETA ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / max(rope, 1))).float()


def _pool(g, batch, capacity, page, dim, dtype):
    """A page pool, more pages than the sequences need, and their table in shuffled order."""
    per = (capacity + page - 1) // page
    n_pages = batch * per + 3
    table = torch.randperm(n_pages, generator=g, device="cuda")[:batch * per].reshape(batch, per).to(torch.int32).contiguous()
    data = _normal(g, n_pages, page, dim, dtype=dtype)
    return data, table


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op = DT[case["dtype"]], case["op"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case)
    if op == "norm_rope":
        n, dim = case["n"], case["dim"]
        # queries and keys as a fused projection leaves them: heads side by side in one row
        x = _normal(g, n, (case["hq"] + case["hk"]) * dim, dtype=dt)
        s["q"] = x[:, :case["hq"] * dim].unflatten(1, (case["hq"], dim))
        s["k"] = x[:, case["hq"] * dim:].unflatten(1, (case["hk"], dim)) if case["hk"] else None
        s["gq"], s["gk"] = (1 + 0.2 * _normal(g, dim) for _ in range(2))
        s["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case["rope"])
        s["out_q"] = torch.empty(n, case["hq"], dim, dtype=dt, device="cuda")
        s["out_k"] = torch.empty(n, case["hk"], dim, dtype=dt, device="cuda") if case["hk"] else None
    elif op == "append":
        b, T, dim = case["batch"], case["T"], case["d_v"] + case["rope"]
        s["data"], s["table"] = _pool(g, b, case["hi"] + T, case["page"], dim, dt)
        s["x"] = _normal(g, b, T, dim, dtype=dt)
        s["gamma"] = 1 + 0.2 * _normal(g, case["d_v"])
        s["start"], s["n_new"] = i32(_lengths(case)), i32(_new(case))
        s["lengths"] = s["start"].clone()
        s["inv_freq"] = _inv_freq(case["rope"])
    elif op == "latent":
        b, T, dim, k = case["batch"], case["T"], case["d_v"] + case["rope"], case["k"]
        lens = _lengths(case)
        s["data"], s["table"] = _pool(g, b, max(case["hi"], 1), case["page"], dim, dt)
        s["lengths"] = i32(lens)
        # scores of a spread that a trained model has: a few positions carry most of the weight
        s["q"] = _normal(g, b, T, case["H"], dim, dtype=dt, scale=2.0)
        s["scale"] = dim ** -0.5
        # the T queries are the last T positions of their sequence
        s["q_pos"] = (s["lengths"][:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32)) if T > 1 else None
        s["sel"] = None
        if k:
            n = s["lengths"][:, None].expand(b, T) if T == 1 else s["q_pos"] + 1
            cap = max(case["hi"], 1)
            r = torch.rand(b, T, cap, generator=g, device="cuda")
            r = torch.where(torch.arange(cap, device="cuda") < n[..., None], r, -1.0)
            v, i = r.topk(min(k, cap), dim=-1)
            i = torch.where(v >= 0, i, cap).sort(-1).values
            i = torch.where(i < cap, i, -1).to(torch.int32)
            s["sel"] = torch.nn.functional.pad(i, (0, k - i.shape[-1]), value=-1).contiguous()
        s["out"] = torch.empty(b, T, case["H"], case["d_v"], dtype=dt, device="cuda")
        s["lse"] = torch.empty(b, T, case["H"], device="cuda")
    else:
        nq = _lengths(case)
        nk = [n + case["past"] for n in nq]
        H = case["H"]
        s["cu_q"], s["cu_k"] = i32([0] + np.cumsum(nq).tolist()), i32([0] + np.cumsum(nk).tolist())
        s["max_q"], s["max_k"] = max(nq), max(nk)
        s["q"] = _normal(g, sum(nq), H, case["nope"] + case["rope"], dtype=dt, scale=2.0)
        # one product expands the latent into every head's keys and values, side by side
        kv = _normal(g, sum(nk), H, case["nope"] + case["d_v"], dtype=dt)
        s["k_nope"], s["v"] = kv[..., :case["nope"]], kv[..., case["nope"]:]
        s["k_rope"] = _normal(g, sum(nk), case["rope"], dtype=dt) if case["rope"] else None
        s["scale"] = (case["nope"] + case["rope"]) ** -0.5
        s["out"] = torch.empty(sum(nq), H, case["d_v"], dtype=dt, device="cuda")
        s["lse"] = torch.empty(sum(nq), H, device="cuda")
    return s


_ctx = None


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # the context, the workspace and the argument records that a serving program keeps
        global _ctx
        import cross_layer_latent_b200 as li
        if _ctx is None:
            _ctx = li.Context(torch.cuda.current_device())
        s["li"], s["ctx"] = li, _ctx
        if case["op"] == "norm_rope":
            tf = [li.RowTransform(norm="rms", norm_dim=case["dim"], gamma=gm, eps=EPS, rope_offset=case["dim"] - case["rope"],
                                  rope_dim=case["rope"], inv_freq=s["inv_freq"], rope_halves=case["halves"])
                  for gm in (s["gq"], s["gk"])]
            s["rows"] = [li.HeadRows(s["q"], tf[0], s["out_q"])]
            if s["k"] is not None:
                s["rows"].append(li.HeadRows(s["k"], tf[1], s["out_k"]))
        elif case["op"] == "append":
            s["tf"] = li.RowTransform(norm="rms", norm_dim=case["d_v"], gamma=s["gamma"], eps=EPS, rope_offset=case["d_v"],
                                      rope_dim=case["rope"], inv_freq=s["inv_freq"])
        if case["op"] in ("append", "latent"):
            s["cache"] = li.PagedCache(s["data"], s["table"], s["lengths"])
        s["ws"] = li.attention_workspace(_ctx, case.get("H", 1), case.get("d_v", 1))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    return (_calls if own else _plain)[case["op"]](s)


def _call_norm_rope(s):
    s["li"].li_norm_rope(s["ctx"], s["rows"], s["pos"])
    return [r.out for r in s["rows"]]


def _call_append(s):
    s["li"].li_append_paged(s["ctx"], s["cache"], s["x"], s["ws"], tf=s["tf"], start=s["start"], n_new=s["n_new"])
    return [s["data"], s["lengths"]]


def _call_latent(s):
    s["li"].li_latent_attention(s["ctx"], s["cache"], s["q"], s["case"]["d_v"], s["scale"], s["out"], s["ws"], lse=s["lse"],
                                sel=s["sel"], q_pos=s["q_pos"])
    return [s["out"], s["lse"]]


def _call_prompt(s):
    s["li"].li_prompt_attention(s["ctx"], s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["scale"],
                                s["out"], s["ws"], lse=s["lse"], causal=True)
    return [s["out"], s["lse"]]


_calls = dict(norm_rope=_call_norm_rope, append=_call_append, latent=_call_latent, prompt=_call_prompt)


# ------------------------------------------------------------------ the plain forms

def _rms(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma


def _rotate(x, pos, inv_freq, halves):
    """x [..., rope] turned by its position; the angle in 64 bits, far positions lose it in 32."""
    a = pos.double()[..., None] * inv_freq.double()
    c, s = a.cos().float(), a.sin().float()
    if halves:
        u, v = x.chunk(2, dim=-1)
        return torch.cat([u * c - v * s, u * s + v * c], dim=-1)
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], dim=-1).flatten(-2)


def _norm_rope(x, gamma, s):
    case = s["case"]
    y = _rms(x.float(), gamma)
    if case["rope"]:
        a = case["dim"] - case["rope"]
        y = torch.cat([y[..., :a], _rotate(y[..., a:], s["pos"][:, None], s["inv_freq"], case["halves"])], dim=-1)
    return y.to(x.dtype)


def _plain_norm_rope(s):
    out = [_norm_rope(s["q"], s["gq"], s)]
    if s["k"] is not None:
        out.append(_norm_rope(s["k"], s["gk"], s))
    return out


def _plain_append(s):
    case = s["case"]
    d_v, T, page = case["d_v"], case["T"], case["page"]
    t = torch.arange(T, device="cuda")
    pos = s["start"][:, None] + t
    x = s["x"].float()
    y = _rms(x[..., :d_v], s["gamma"])
    if case["rope"]:
        y = torch.cat([y, _rotate(x[..., d_v:], pos, s["inv_freq"], False)], dim=-1)
    live = t < s["n_new"][:, None]
    at = torch.where(live, pos, 0).long()
    row = s["table"].long().gather(1, at // page) * page + at % page
    s["data"].flatten(0, 1)[row[live]] = y[live].to(s["data"].dtype)
    s["lengths"].copy_(s["start"] + s["n_new"])
    return [s["data"], s["lengths"]]


def _softmax_sums(score, live):
    """Weights, their sums and the log of those, of scores [..., n]; a row with nothing live has weights 0 and -inf."""
    score = torch.where(live, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = (score - m).exp()
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, 1.0), (m + total.log())[..., 0]


def _plain_latent(s):
    case = s["case"]
    b, T, page = case["batch"], case["T"], case["page"]
    n = s["lengths"][:, None].expand(b, T)
    if s["q_pos"] is not None:
        n = torch.minimum(n, s["q_pos"] + 1)
    flat = s["data"].flatten(0, 1)
    table = s["table"].long()
    if s["sel"] is None:
        at = torch.arange(max(case["hi"], 1), device="cuda").expand(b, -1)
        live = (at[:, None] < n[..., None])[:, :, None]
        rows = flat[table.gather(1, at // page) * page + at % page].float()[:, None]
    else:
        live = (s["sel"] >= 0) & (s["sel"] < n[..., None])
        at = torch.where(live, s["sel"], 0).long().flatten(1)
        rows = flat[table.gather(1, at // page) * page + at % page].float().unflatten(1, (T, -1))
        live = live[:, :, None]
    score = s["q"].float() @ rows.transpose(-1, -2) * s["scale"]
    p, total, lse = _softmax_sums(score, live)
    return [((p @ rows[..., :case["d_v"]]) / total).to(s["q"].dtype), lse]


def _padded(x, cu, width):
    """Rows of a ragged batch as [batch, width, ...], and which of them are there."""
    n = (cu[1:] - cu[:-1])[:, None]
    t = torch.arange(width, device="cuda")
    there = t < n
    return x[torch.where(there, cu[:-1, None] + t, 0).long()], there


def _plain_prompt(s):
    q, there_q = _padded(s["q"].float(), s["cu_q"], s["max_q"])
    k, there_k = _padded(s["k_nope"].float(), s["cu_k"], s["max_k"])
    v, _ = _padded(s["v"].float(), s["cu_k"], s["max_k"])
    if s["k_rope"] is not None:
        r, _ = _padded(s["k_rope"].float(), s["cu_k"], s["max_k"])
        k = torch.cat([k, r[:, :, None].expand(-1, -1, k.shape[2], -1)], dim=-1)
    nq, nk = (c[1:] - c[:-1] for c in (s["cu_q"], s["cu_k"]))
    i, j = torch.arange(s["max_q"], device="cuda"), torch.arange(s["max_k"], device="cuda")
    live = there_k[:, None] & (j <= i[:, None] + (nk - nq)[:, None, None])
    score = q.transpose(1, 2) @ k.permute(0, 2, 3, 1) * s["scale"]
    p, total, lse = _softmax_sums(score, live[:, None])
    out = (p @ v.transpose(1, 2)) / total
    return [out.transpose(1, 2)[there_q].to(s["q"].dtype), lse.transpose(1, 2)[there_q].contiguous()]


_plain = dict(norm_rope=_plain_norm_rope, append=_plain_append, latent=_plain_latent, prompt=_plain_prompt)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "norm_rope":
        rows = case["n"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * rows * case["dim"] * e + 4 * case["n"] + 8 * case["dim"], "flops": rows * (4 * case["dim"] + 3 * case["rope"])}
    if op == "append":
        n, dim = sum(_new(case)), case["d_v"] + case["rope"]
        return {"bytes": 2 * n * dim * e + 4 * case["d_v"], "flops": n * (4 * case["d_v"] + 3 * case["rope"])}
    if op == "latent":
        b, T, H, d_v, dim, k = case["batch"], case["T"], case["H"], case["d_v"], case["d_v"] + case["rope"], case["k"]
        pairs = rows = sels = 0
        for n in _lengths(case):
            per = [max(0, n - T + 1 + t) for t in range(T)]
            per = [min(k, x) for x in per] if k else per
            pairs, rows = pairs + sum(per), rows + min(n, sum(per))
            sels += 4 * k * T
        return {"bytes": rows * dim * e + sels + b * T * H * ((dim + d_v) * e + 4), "flops": max(1, 2 * H * pairs * (dim + d_v))}
    nq = _lengths(case)
    dk, d_v, H = case["nope"] + case["rope"], case["d_v"], case["H"]
    pairs = sum(n * (case["past"] + (n + 1) / 2) for n in nq)
    nk = sum(nq) + case["past"] * len(nq)
    return {"bytes": e * H * (sum(nq) * (dk + d_v) + nk * (case["nope"] + d_v)) + e * nk * case["rope"] + 4 * H * sum(nq),
            "flops": max(1, int(2 * H * pairs * (dk + d_v)))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _turn64(x, pos, rope, halves):
    """Complex multiplication by exp(i pos f) of the rotary slots, one frequency a slot."""
    f = torch.from_numpy(np.power(THETA, -np.arange(0, rope, 2) / rope).astype(np.float32).astype(np.float64)).to(x.device)
    w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.to(torch.float64)[..., None] * f)
    half = rope // 2
    z = torch.complex(x[..., :half], x[..., half:]) if halves else torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous())
    z = z * w
    return torch.cat([z.real, z.imag], -1) if halves else torch.view_as_real(z).reshape(x.shape)


def _unit64(x, gamma):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gamma.to(torch.float64)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm_rope":
        out = []
        for x, gamma in ((s["q"], s["gq"]), (s["k"], s["gk"])):
            if x is not None:
                y, r = _unit64(x.double(), gamma), case["rope"]
                if r:
                    y[..., case["dim"] - r:] = _turn64(y[..., case["dim"] - r:].clone(), s["pos"][:, None], r, case["halves"])
                out.append(y)
        return out
    if op == "append":
        data = s["data"].double()
        for b, (at, n) in enumerate(zip(_lengths(case), _new(case))):
            x = s["x"][b, :n].double()
            p = torch.arange(at, at + n, device="cuda")
            y = x.clone()
            y[:, :case["d_v"]] = _unit64(x[:, :case["d_v"]], s["gamma"])
            if case["rope"]:
                y[:, case["d_v"]:] = _turn64(x[:, case["d_v"]:], p, case["rope"], False)
            data[s["table"][b, p // case["page"]].long(), p % case["page"]] = y
        return [data, s["start"] + s["n_new"]]
    if op == "latent":
        if work(case)["flops"] > 4e11:
            return None
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            for t in range(case["T"]):
                m = n - case["T"] + 1 + t
                p = torch.arange(max(m, 0), device="cuda") if s["sel"] is None else s["sel"][b, t][s["sel"][b, t] >= 0].long()
                if len(p):
                    c = s["data"][s["table"][b, p // case["page"]].long(), p % case["page"]].double()
                    z = s["scale"] * (s["q"][b, t].double() @ c.T)
                    lse[b, t] = torch.logsumexp(z, -1)
                    out[b, t] = torch.softmax(z, -1) @ c[:, :case["d_v"]]
        return [out, lse]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n in _lengths(case):
        m = n + case["past"]
        for h in range(case["H"]):
            k = s["k_nope"][k0:k0 + m, h].double()
            if s["k_rope"] is not None:
                k = torch.cat([k, s["k_rope"][k0:k0 + m].double()], -1)
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                last = torch.arange(r, e, device="cuda")[:, None] + case["past"]
                z = s["scale"] * (s["q"][q0 + r:q0 + e, h].double() @ k.T)
                z = z.masked_fill(torch.arange(m, device="cuda") > last, -math.inf)
                lse[q0 + r:q0 + e, h] = torch.logsumexp(z, -1)
                out[q0 + r:q0 + e, h] = torch.softmax(z, -1) @ s["v"][k0:k0 + m, h].double()
        q0, k0 = q0 + n, k0 + m
    return [out, lse]
