"""Measured cases of the operators that choose from a vocabulary, learn from what was chosen, and the 8-bit head.

Each in a plain form (elementary torch operations in fp32, in fp64 where fp32
loses what matters) and, where `own` is true, through this package's entry
points:

* top      -- the K largest logits of a row with their log-probs, the mass of all others and the log-sum-exp (what a
              teacher leaves behind for distillation, or a server returns beside a token);
* distill  -- KL from such a teacher's list to a student's whole row, and distill_grad its gradient with respect to
              the student's logits;
* beam     -- the best N continuations over beams and vocabulary, and reorder the states that follow their beams;
* fp8      -- logits through an output head held in 8-bit floats with a scale for each block of 128 x 128, the hidden
              rows brought to 8 bits with a scale for each 128 columns on the way.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEG_INF = float("-inf")
BLOCK = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the alternatives that a server returns beside one decoded token
        dict(name="top_one_row", kind="top", dtype="bf16", T=1, V=151936, K=20, tau=1.0, mask=False),
        # a teacher's pass over a packed batch, prompt rows left out
        dict(name="top_teacher", kind="top", dtype="bf16", T=8192, V=151936, K=64, tau=1.0, mask=True),
        # a handful of odd fp32 rows, lists without the mass of the others
        dict(name="distill_odd_rows", kind="distill", dtype="fp32", T=5, V=20011, K=17, tau=1.3, mask=False, rest=False),
        # the student's loss over a packed batch
        dict(name="distill_batch", kind="distill", dtype="bf16", T=8192, V=151936, K=64, tau=1.0, mask=True, rest=True),
        # the gradient of a small ragged batch
        dict(name="distill_grad_small", kind="distill_grad", dtype="fp16", T=37, V=4099, K=32, tau=1.3, mask=False,
             rest=True),
        # the gradient of one training step
        dict(name="distill_grad_batch", kind="distill_grad", dtype="bf16", T=4096, V=151936, K=64, tau=1.0, mask=False,
             rest=True),
        # one request decoded with four beams, twice as many continuations asked for as beams go on
        dict(name="beam_one_request", kind="beam", dtype="bf16", B=1, W=4, V=151936, N=8, tau=1.0, finished=False),
        # a full decode batch of eight beams, some of them finished
        dict(name="beam_batch", kind="beam", dtype="fp16", B=64, W=8, V=129280, N=16, tau=1.0, finished=True),
        # token histories of a decode batch follow their beams
        dict(name="reorder_histories", kind="reorder", dtype="int32", outer=1, B=32, W=8, N=8, mid=1, used=1517, cap=2048),
        # caches of 48 layers follow their beams: of each row the positions in use
        dict(name="reorder_cache", kind="reorder", dtype="bf16", outer=48, B=32, W=8, N=8, mid=1, used=128 * 1001,
             cap=128 * 1024),
        # the head of a small decode batch
        dict(name="fp8_decode", kind="fp8", dtype="bf16", out="fp32", T=8, h=5120, V=151936),
        # a teacher's head over a batch of rows
        dict(name="fp8_teacher", kind="fp8", dtype="bf16", out="bf16", T=4096, h=7168, V=129280),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["top", "distill", "distill_grad", "beam", "reorder", "fp8", "fp8"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    tau = rng.choice([1.0, 1.0, 0.7, rng.uniform(0.5, 2.0)])
    if kind in ("top", "distill", "distill_grad"):
        most = {"top": 8192, "distill": 8192, "distill_grad": 4096}[kind]
        c = dict(kind=kind, dtype=dtype, T=_spread(rng, 1, most if dtype != "fp32" else most // 2),
                 V=_spread(rng, 1000, 151936), K=_spread(rng, 1, 256), tau=tau, mask=rng.random() < 0.5)
        if kind != "top":
            c["rest"] = rng.random() < 0.7
        return c
    if kind == "beam":
        W = rng.choice([1, 2, 3, 4, 5, 8, 10])
        return dict(kind=kind, dtype=dtype, B=_spread(rng, 1, 512 // W if dtype != "fp32" else 256 // W), W=W,
                    V=_spread(rng, 1000, 129280), N=rng.choice([W, 2 * W]), tau=tau, finished=rng.random() < 0.5)
    if kind == "reorder":
        W = rng.choice([2, 3, 4, 5, 8])
        dtype = rng.choice(["int32", "bf16", "fp32", "fp16"])
        outer = 1 if dtype == "int32" else _spread(rng, 1, 48)
        used = _spread(rng, 1, 2048) if dtype == "int32" else rng.choice([64, 80, 128]) * _spread(rng, 1, 500)
        return dict(kind=kind, dtype=dtype, outer=outer, B=_spread(rng, 1, 32), W=W, N=W,
                    mid=1 if dtype == "int32" else rng.choice([1, 2, 3]), used=used, cap=used + rng.randint(0, used // 2))
    return dict(kind=kind, dtype=rng.choice(["bf16", "fp16"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                T=_spread(rng, 1, 4096), h=16 * _spread(rng, 8, 448), V=_spread(rng, 100, 129280))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _scored(T):
    """Rows that are scored where a case has a mask: three of four, in short runs."""
    return torch.arange(T, device="cuda") % 16 >= 4


def _scored_rows(c):
    return sum(1 for t in range(c["T"]) if t % 16 >= 4) if c["mask"] else c["T"]


def _logits(T, V, gen, dt):
    """Rows as a trained model gives them: a broad floor, and some tens of columns well above it."""
    z = torch.randn(T, V, generator=gen, device="cuda").mul_(2.0)
    n = min(48, V)
    at = torch.randint(0, V, (T, n), generator=gen, device="cuda")
    up = 4.0 + 10.0 * torch.rand(T, n, generator=gen, device="cuda")
    return z.scatter_add_(1, at, up).to(dt)


def _teacher(c, s, gen):
    """Lists of a teacher near the student: ids, log-probs, and the log of the mass left; one row in eight is short."""
    T, V, K = c["T"], c["V"], min(c["K"], c["V"])
    s["ids"] = torch.empty(T, K, dtype=torch.int64, device="cuda")
    s["logprob"] = torch.empty(T, K, device="cuda")
    s["rest"] = torch.empty(T, device="cuda") if c["rest"] else None
    part = max(1, (1 << 28) // V)
    for r in range(0, T, part):
        z = s["logits"][r:r + part].float()
        z = (z + 0.5 * torch.randn(z.shape, generator=gen, device="cuda")) / c["tau"]
        top, s["ids"][r:r + part] = z.topk(K, 1)
        lse = torch.logsumexp(z, 1)
        s["logprob"][r:r + part] = top - lse[:, None]
        if c["rest"]:
            z.scatter_(1, s["ids"][r:r + part], NEG_INF)
            s["rest"][r:r + part] = torch.logsumexp(z, 1) - lse
    if K > 2:
        short = torch.arange(T, device="cuda") % 8 == 5
        s["ids"][short, K - 2:] = -1
        s["logprob"][short, K - 2:] = NEG_INF


def _beams(c, s, gen):
    """Scores so far, apart enough that which continuation is better does not hang on a rounding."""
    B, W, V, N = c["B"], c["W"], c["V"], c["N"]
    s["logits"] = _logits(B * W, V, gen, DTYPES[c["dtype"]])
    s["beam_scores"] = -20.0 * torch.rand(B, W, generator=gen, device="cuda").sort(1)[0]
    s["finished"] = None
    if c["finished"]:
        s["finished"] = torch.rand(B, W, generator=gen, device="cuda") < 0.15
    elif W > 1:
        # a request that has just begun: one beam goes on, the others are empty
        s["beam_scores"][::4, 1:] = NEG_INF
    n = min(N + 1, V)
    top, lse = [], []
    for z in s["logits"].split(max(1, (1 << 27) // V)):
        z = z.double() / c["tau"]
        top.append(z.topk(n, 1)[0])
        lse.append(torch.logsumexp(z, 1))
    gain = (torch.cat(top) - torch.cat(lse)[:, None]).view(B, W, n)
    if c["finished"]:
        gain = torch.where(s["finished"][:, :, None], NEG_INF, gain)
        gain[:, :, 0] = torch.where(s["finished"], 0.0, gain[:, :, 0])
    beam = torch.arange(W, device="cuda").repeat_interleave(n).expand(B, -1)
    for _ in range(50):
        score, order = (s["beam_scores"].double()[:, :, None] + gain).flatten(1).sort(1, descending=True)
        who = beam.gather(1, order)
        near = (score[:, :-1] - score[:, 1:] < 1e-4) & (who[:, :-1] != who[:, 1:]) & (score[:, 1:] > NEG_INF)
        near = near[:, :2 * N].any(1)
        s["beam_scores"] -= near[:, None] * torch.rand(B, W, generator=gen, device="cuda")


def _parents(c, gen):
    """Beams that go on: five of eight of them, some more than once."""
    B, W, N = c["B"], c["W"], c["N"]
    keep = max(1, W * 5 // 8)
    who = torch.rand(B, W, generator=gen, device="cuda").argsort(1)[:, :keep]
    slot = torch.arange(N, device="cuda") % keep
    mix = torch.rand(B, N, generator=gen, device="cuda").argsort(1)
    return who.gather(1, slot[mix]).int()


def prepare(case, seed):
    c, kind = case, case["kind"]
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    s = {"case": c}
    if kind in ("top", "distill", "distill_grad"):
        s["logits"] = _logits(c["T"], c["V"], gen, DTYPES[c["dtype"]])
        s["mask"] = _scored(c["T"]) if c["mask"] else None
        if kind != "top":
            _teacher(c, s, gen)
        if kind == "distill_grad":
            # what the forward left
            _, s["lse"], s["lse_rest"] = _plain_distill(s)
            s["grad_loss"] = 1.0 / c["T"] * (0.5 + torch.rand(c["T"], generator=gen, device="cuda"))
        return s
    if kind == "beam":
        _beams(c, s, gen)
        return s
    if kind == "reorder":
        shape = (c["outer"], c["B"] * c["W"], c["mid"], c["cap"])
        if c["dtype"] == "int32":
            whole = torch.randint(0, 1 << 17, shape, generator=gen, device="cuda", dtype=torch.int32)
        else:
            whole = torch.empty(shape, dtype=DTYPES[c["dtype"]], device="cuda")
            for layer in whole:
                layer.normal_(generator=gen)
        s["state"] = whole[..., :c["used"]]
        s["parents"] = _parents(c, gen)
        return s
    T, h, V = c["T"], c["h"], c["V"]
    x = torch.randn(T, h, generator=gen, device="cuda")
    x[:, torch.randint(0, h, (4,), generator=gen, device="cuda")] *= 20.0  # columns that stand out in every row
    s["hidden"] = x.to(DTYPES[c["dtype"]])
    s["weight"] = torch.empty(V, h, dtype=torch.float8_e4m3fn, device="cuda")
    part = max(1, (1 << 28) // h)
    for v in range(0, V, part):
        w = torch.randn(min(part, V - v), h, generator=gen, device="cuda").mul_(110.0).clamp_(-448.0, 448.0)
        s["weight"][v:v + part] = w.to(torch.float8_e4m3fn)
    blocks = (-(-V // BLOCK), -(-h // BLOCK))
    s["scales"] = 0.0002 * (0.5 + torch.rand(blocks, generator=gen, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rank_keys(z):
    """Whole numbers in the order of the values of z [R, V], of equal ones the lowest column first."""
    bits = (z.float() + 0.0).view(torch.int32).long()
    bits = torch.where(bits < 0, -1 - (bits & 0x7fffffff), bits)
    return (bits << 30) - torch.arange(z.shape[1], device=z.device)


def _plain_top(s):
    c = s["case"]
    T, V, K = c["T"], c["V"], min(c["K"], c["V"])
    ids = torch.full((T, K), -1, dtype=torch.int64, device="cuda")
    logprob, rest, lse = torch.zeros(T, K, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    rows = torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0]
    for r in rows.split(max(1, (1 << 29) // V)):
        raw = s["logits"] if s["mask"] is None and r.numel() == T else s["logits"][r]
        pick = _rank_keys(raw).topk(K, 1)[1]
        z = raw.float() / c["tau"]
        m = z.amax(1)
        whole = m + (z - m[:, None]).exp().sum(1).log()
        ids[r], lse[r] = pick, whole
        logprob[r] = z.gather(1, pick) - whole[:, None]
        z = z.scatter(1, pick, NEG_INF)
        m = z.amax(1).clamp(min=-1e30)
        rest[r] = m + (z - m[:, None]).exp().sum(1).log() - whole
    return ids, logprob, rest, lse


def _listed(s):
    """(listed columns [T, V], probabilities of the entries [T, K], their log-probs, ids to look up)."""
    c = s["case"]
    ok = (s["ids"] >= 0) & (s["ids"] < c["V"])
    at = torch.where(ok, s["ids"], c["V"])
    listed_ = torch.zeros(c["T"], c["V"] + 1, dtype=torch.bool, device="cuda").scatter_(1, at, True)[:, :c["V"]]
    p = torch.where(ok, s["logprob"].exp(), 0.0)
    return listed_, p, s["logprob"], torch.where(ok, s["ids"], 0)


def _plain_distill(s):
    c = s["case"]
    listed_, p, t, ids = _listed(s)
    z = s["logits"].float() / c["tau"]
    m = z.amax(1, keepdim=True)
    lse = (m + (z - m).exp().sum(1, keepdim=True).log())[:, 0]
    u = z.masked_fill(listed_, NEG_INF)
    m = u.amax(1, keepdim=True).clamp(min=-1e30)
    lse_rest = (m + (u - m).exp().sum(1, keepdim=True).log())[:, 0]
    logq = z.gather(1, ids) - lse[:, None]
    loss = torch.where(p > 0, p * (t - logq), 0.0).sum(1)
    if s["rest"] is not None:
        r = s["rest"].exp()
        loss = loss + torch.where(r > 0, r * (s["rest"] - (lse_rest - lse)), 0.0)
    if s["mask"] is not None:
        loss, lse, lse_rest = (torch.where(s["mask"], x, 0.0) for x in (loss, lse, lse_rest))
    return loss, lse, lse_rest


def _plain_distill_grad(s):
    c = s["case"]
    listed_, p, _, ids = _listed(s)
    z = s["logits"].float() / c["tau"]
    r = torch.zeros_like(s["lse"]) if s["rest"] is None else s["rest"].exp()
    whole = p.sum(1) + r
    rq = (s["lse_rest"] - s["lse"]).exp()
    d = torch.where(listed_, (z - s["lse"][:, None]).exp() * whole[:, None],
                    (z - s["lse_rest"][:, None]).exp() * (whole * rq - r)[:, None])
    d.scatter_add_(1, ids, -p)
    d *= (s["grad_loss"] / c["tau"])[:, None]
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None], d, 0.0)
    return d.to(s["logits"].dtype)


def _plain_beam(s):
    c = s["case"]
    B, W, V, N = c["B"], c["W"], c["V"], c["N"]
    n = min(N, V)
    pick, gain = [], []
    for raw in s["logits"].split(max(1, (1 << 28) // V)):
        k = _rank_keys(raw).topk(n, 1)[1]
        z = raw.double() / c["tau"]
        m = z.amax(1, keepdim=True)
        pick.append(k)
        gain.append(z.gather(1, k) - m - (z - m).exp().sum(1, keepdim=True).log())
    pick, gain = torch.cat(pick).view(B, W, n), torch.cat(gain).view(B, W, n)
    if s["finished"] is not None:
        first = torch.arange(n, device="cuda") == 0
        gain = torch.where(s["finished"][:, :, None], torch.where(first, 0.0, NEG_INF), gain)
        pick = torch.where(s["finished"][:, :, None], END, pick)
    score = (s["beam_scores"].double()[:, :, None] + gain).flatten(1)
    score, order = score.sort(dim=1, descending=True, stable=True)
    short = max(0, N - W * n)
    score, order = score[:, :N], order[:, :N]
    live = score > NEG_INF
    tokens = torch.where(live, pick.flatten(1).gather(1, order), -1)
    parents = torch.where(live, order // n, -1).int()
    pad = torch.nn.functional.pad
    return pad(score.float(), (0, short), value=NEG_INF), pad(parents, (0, short), value=-1), pad(tokens, (0, short), value=-1)


def _plain_reorder(s):
    c = s["case"]
    at = (torch.arange(c["B"], device="cuda")[:, None] * c["W"] + s["parents"]).flatten()
    return s["state"][:, at]


def _to_blocks(x):
    """x [R, h] as [R, blocks, 128], zeros behind the last column."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))


def _plain_fp8(s):
    c = s["case"]
    x = _to_blocks(s["hidden"].float())
    sx = (x.abs().amax(2, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
    x = ((x / sx).to(torch.float8_e4m3fn).float() * sx).flatten(1)[:, :c["h"]]
    out = torch.empty(c["T"], c["V"], dtype=DTYPES[c["out"]], device="cuda")
    part = max(BLOCK, (1 << 29) // c["h"] // BLOCK * BLOCK)
    for v in range(0, c["V"], part):
        w = s["weight"][v:v + part].float()
        scale = s["scales"][v // BLOCK:(v + part) // BLOCK].repeat_interleave(BLOCK, 1)[:, :c["h"]]
        w = w * scale.repeat_interleave(BLOCK, 0)[:w.shape[0]]
        out[:, v:v + part] = x @ w.t()
    return out


END = 2  # the token that ends a sequence


def _plain(s):
    kind = s["case"]["kind"]
    return {"top": _plain_top, "distill": _plain_distill, "distill_grad": _plain_distill_grad, "beam": _plain_beam,
            "reorder": _plain_reorder, "fp8": _plain_fp8}[kind](s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import entropy_chunked_row_amd as lp

    c, kind = s["case"], s["case"]["kind"]
    if kind == "top":
        return lp.lp_top_logits(s["logits"], min(c["K"], c["V"]), s["mask"], c["tau"])
    if kind == "distill":
        return lp.lp_distill_top(s["logits"], s["ids"], s["logprob"], s["rest"], s["mask"], c["tau"])
    if kind == "distill_grad":
        return lp.lp_distill_top_backward(s["logits"], s["ids"], s["logprob"], s["rest"], s["mask"], c["tau"], s["lse"],
                                          s["lse_rest"], s["grad_loss"])
    if kind == "beam":
        return lp.lp_beam_select(s["logits"], s["beam_scores"], c["N"], s["finished"], END, c["tau"])
    if kind == "reorder":
        return lp.lp_beam_reorder(s["state"], s["parents"], dim=1)
    return lp.lp_lm_head_fp8_logits(s["hidden"], s["weight"], s["scales"], out_dtype=DTYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, kind = case, case["kind"]
    size = 4 if c["dtype"] in ("fp32", "int32") else 2
    if kind in ("top", "distill", "distill_grad"):
        T, V, K = c["T"], c["V"], min(c["K"], c["V"])
        n = _scored_rows(c)
        if kind == "top":
            return {"bytes": n * V * size + T * (12 * K + 8), "flops": 4 * n * V}
        lists = n * (12 * K + 4)
        if kind == "distill":
            return {"bytes": n * V * size + lists + 12 * T, "flops": 4 * n * V}
        return {"bytes": (n + T) * V * size + lists + 12 * n, "flops": 5 * n * V}
    if kind == "beam":
        n = c["B"] * c["W"]
        return {"bytes": n * c["V"] * size + 5 * n + 16 * c["B"] * c["N"], "flops": 4 * n * c["V"]}
    if kind == "reorder":
        row = c["outer"] * c["mid"] * c["used"] * size
        return {"bytes": row * c["B"] * (min(c["N"], max(1, c["W"] * 5 // 8)) + c["N"]) + 4 * c["B"] * c["N"], "flops": 0}
    T, h, V = c["T"], c["h"], c["V"]
    out = 4 if c["out"] == "fp32" else 2
    scales = 4 * -(-V // BLOCK) * -(-h // BLOCK)
    return {"bytes": V * h + scales + T * (h * size + V * out), "flops": 2 * T * h * V}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _order(z):
    """Columns of one row from its largest value down, equal ones from the lowest column up."""
    return torch.argsort(z, descending=True, stable=True)


def _exact_top(c, s, t):
    z = s["logits"][t].double()
    at = _order(z)
    z = z / c["tau"]
    K = min(c["K"], c["V"])
    lse = torch.logsumexp(z, 0)
    return at[:K], z[at[:K]] - lse, torch.logsumexp(z[at[K:]], 0) - lse, lse


def _exact_entries(c, s, t):
    ids, lp = s["ids"][t], s["logprob"][t].double()
    keep = (ids >= 0) & (ids < c["V"]) & (lp > NEG_INF)
    inside = ids[(ids >= 0) & (ids < c["V"])]
    other = torch.ones(c["V"], dtype=torch.bool, device="cuda")
    other[inside] = False
    return ids[keep], lp[keep], other


def _exact_distill(c, s, t):
    ids, lp, other = _exact_entries(c, s, t)
    z = s["logits"][t].double() / c["tau"]
    lse, lse_rest = torch.logsumexp(z, 0), torch.logsumexp(z[other], 0)
    loss = (lp.exp() * (lp - (z[ids] - lse))).sum()
    if s["rest"] is not None and s["rest"][t] > NEG_INF:
        r = s["rest"][t].double()
        loss = loss + r.exp() * (r - (lse_rest - lse))
    return loss, lse, lse_rest


def _exact_distill_grad(c, s, t):
    ids, lp, other = _exact_entries(c, s, t)
    z = s["logits"][t].double() / c["tau"]
    lse, lse_rest = s["lse"][t].double(), s["lse_rest"][t].double()
    r = s["rest"][t].double().exp() if s["rest"] is not None else torch.zeros((), dtype=torch.float64, device="cuda")
    mass = lp.exp().sum() + r
    # of each listed column its own share, of the others their part of one shared share
    d = mass * torch.softmax(z, 0) * (torch.logsumexp(z, 0) - lse).exp()
    d[other] = (z[other] - lse_rest).exp() * (mass * (lse_rest - lse).exp() - r)
    d.index_add_(0, ids, -lp.exp())
    return d * s["grad_loss"][t].double() / c["tau"]


def _exact_beam(c, s):
    B, W, V, N = c["B"], c["W"], c["V"], c["N"]
    scores, parents, tokens = [], [], []
    for b in range(B):
        z = s["logits"][b * W:(b + 1) * W].double() / c["tau"]
        z = z - torch.logsumexp(z, 1, keepdim=True) + s["beam_scores"][b].double()[:, None]
        for w in range(W):
            if s["finished"] is not None and bool(s["finished"][b, w]):
                z[w] = NEG_INF
                z[w, END] = s["beam_scores"][b, w].double()
        z = z.flatten()
        at = _order(z)[:N]
        z = z[at]
        live = z > NEG_INF
        miss = N - at.numel()
        put = lambda x, v: torch.cat([x, x.new_full((miss,), v)])  # noqa: E731
        scores.append(put(z, NEG_INF))
        parents.append(put(torch.where(live, at // V, -1), -1))
        tokens.append(put(torch.where(live, at % V, -1), -1))
    return torch.stack(scores), torch.stack(parents).int(), torch.stack(tokens)


def _exact_fp8(c, s):
    x, h = s["hidden"].float(), c["h"]
    out = torch.zeros(c["T"], c["V"], dtype=torch.float64, device="cuda")
    row = torch.arange(c["V"], device="cuda") // BLOCK
    for b, k in enumerate(range(0, h, BLOCK)):
        xb = x[:, k:k + BLOCK]
        # the scale and the quotient are fp32 numbers by definition, the product and the sum are not rounded
        step = torch.clamp(xb.abs().max(1, keepdim=True)[0] / 448.0, min=2.0 ** -126)
        q = (xb / step).to(torch.float8_e4m3fn).double()
        dot = q @ s["weight"][:, k:k + BLOCK].double().t()
        out += dot * step.double() * s["scales"][:, b].double()[row]
    return out


def _exact_reorder(c, s):
    src = s["state"].double() if s["state"].is_floating_point() else s["state"]
    parts = src.split(c["W"], 1)
    return torch.cat([part.index_select(1, at.long()) for part, at in zip(parts, s["parents"])], 1)


def exact(case, seed):
    c, kind = case, case["kind"]
    if kind == "fp8" and 2 * c["T"] * c["h"] * c["V"] > 3e14:
        return None
    s = prepare(case, seed)
    if kind == "reorder":
        return _exact_reorder(c, s) if s["state"].numel() <= 1 << 28 else None
    if kind == "beam":
        return _exact_beam(c, s)
    if kind == "fp8":
        return _exact_fp8(c, s)
    if kind == "distill_grad" and c["T"] * c["V"] > 1 << 30:
        return None
    K = min(c["K"], c["V"])
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    rows = []
    for t in range(c["T"]):
        if s["mask"] is not None and not bool(s["mask"][t]):
            none = {"top": (torch.full((K,), -1, device="cuda"), zero.expand(K), zero, zero), "distill": (zero, zero, zero),
                    "distill_grad": zero.expand(c["V"])}
            rows.append(none[kind])
        else:
            rows.append({"top": _exact_top, "distill": _exact_distill, "distill_grad": _exact_distill_grad}[kind](c, s, t))
    if kind == "distill_grad":
        return torch.stack(rows)
    return tuple(torch.stack(x) for x in zip(*rows))
