"""Low-rank adapters beside the NVFP4 projections, and activations kept in 8 bits for their gradients.

A projection's frozen weights are shared by all requests; a request's adapter g adds scale[g] (x a_g^T) b_g to its rows.
Both factors are stored with the rank first: a [adapters, rank, c_in], b [adapters, rank, c_out].  Consecutive rows that
belong together (a request's tokens, an expert's rows) form a segment, and every segment names its adapter, or none (-1).

  lora     y = base + scale (x a^T) b for all segments at once; base is what the shared projection gave
  grad     dx = base + scale (dy b^T) a, its gradient to the input; base is the projection's own
  weights  da = scale (dy b^T)^T x and db = scale (x a^T)^T dy, summed over each adapter's rows; x as it was, or from a
           checkpoint in 8 bits
  pack     a checkpoint of activations: 32 values of a row share a power of two, the smallest with which none exceeds
           448, and are rounded to E4M3
  unpack   the activations back from a checkpoint

`own` selects between the framework's kernels and the plain form, which is elementary torch arithmetic in 32 bits.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
SHARED = 32  # values that share a power of two


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


# ---------------------------------------------------------------------------
# cases: x, w: types of activations and adapters; bare: share of the segments without an adapter; single: every row is a
# segment of its own; kept: what the backward pass has of x ("e4m3": the checkpoint)
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token with one of 8 adapters through the widest projection: a latency
        dict(name="lora-1-mlp-down", kind="lora", rows=1, c_in=17408, c_out=5120, rank=16, adapters=8, segments=1, single=True, bare=0.0, x="bf16", w="bf16"),
        # a decode batch of 48 sequences, each with one of 32 adapters, a few with none
        dict(name="lora-48-mlp-up", kind="lora", rows=48, c_in=4096, c_out=12288, rank=16, adapters=32, segments=48, single=True, bare=0.1, x="bf16", w="bf16"),
        # a prompt batch of 13 requests of all lengths
        dict(name="lora-8192-mlp-up", kind="lora", rows=8192, c_in=4096, c_out=12288, rank=16, adapters=8, segments=13, single=False, bare=0.1, x="bf16", w="bf16"),
        # fp32 activations and adapters of an odd number of tokens
        dict(name="lora-333-dense-f32", kind="lora", rows=333, c_in=4096, c_out=4096, rank=8, adapters=4, segments=5, single=False, bare=0.0, x="f32", w="f32"),
        # training one adapter beside a projection
        dict(name="grad-4096-mlp-up", kind="grad", rows=4096, c_in=4096, c_out=12288, rank=64, adapters=1, segments=1, single=False, bare=0.0, x="bf16", w="bf16"),
        # training an adapter for each of 64 experts, skewed routing
        dict(name="grad-32768-experts", kind="grad", rows=32768, c_in=2048, c_out=1024, rank=16, adapters=64, segments=64, single=False, bare=0.0, x="bf16", w="bf16"),
        # the adapter's own gradients, the activations kept as they were
        dict(name="weights-4096-mlp-up", kind="weights", rows=4096, c_in=4096, c_out=12288, rank=64, adapters=1, segments=1, single=False, bare=0.0, x="bf16", w="bf16", kept="x"),
        # those of the experts' adapters, from a checkpoint in 8 bits
        dict(name="weights-32768-experts-e4m3", kind="weights", rows=32768, c_in=2048, c_out=1024, rank=16, adapters=64, segments=64, single=False, bare=0.0, x="bf16", w="bf16", kept="e4m3"),
        # a few tokens' activations on their way into a checkpoint: a latency
        dict(name="pack-7x4096-f32", kind="pack", rows=7, c_in=4096, x="f32"),
        # a training batch's activations of the widest layer
        dict(name="pack-16384x17408", kind="pack", rows=16384, c_in=17408, x="bf16"),
        # a checkpoint read back for a small layer's backward pass, rows of an odd length
        dict(name="unpack-333x1111-f32", kind="unpack", rows=333, c_in=1111, x="f32"),
        # and for the widest layer's
        dict(name="unpack-16384x17408", kind="unpack", rows=16384, c_in=17408, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly whole blocks of 16, as the projections have them; now and then any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else 16 * max(1, n // 16)


def draw(rng):
    kind = rng.choice(["lora", "lora", "lora", "grad", "grad", "weights", "weights", "pack", "unpack"])
    x = rng.choice(["bf16", "bf16", "f32"])
    c_in = _width(rng, 128, 17408)
    if kind in ("pack", "unpack"):
        rows = _log(rng, 1, 16384)
        while rows * c_in > (1 << 27):
            rows = rows // 2 + 1
        return dict(kind=kind, rows=rows, c_in=c_in, x=x)
    c_out = _width(rng, 128, 17408)
    rank = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 128)])
    single = kind != "weights" and rng.random() < 0.4
    rows = _log(rng, 1, 256 if single else 8192)
    while rows * (c_in + c_out) > 8192 * 8192:
        rows = rows // 2 + 1
    adapters = _log(rng, 1, 64)
    while adapters * rank * (c_in + c_out) > 1 << 25:
        adapters = adapters // 2 + 1
        rank = max(1, rank * 3 // 4)
    segments = rows if single else min(rows, _log(rng, 1, 32))
    case = dict(kind=kind, rows=rows, c_in=c_in, c_out=c_out, rank=rank, adapters=adapters, segments=segments, single=single,
                bare=rng.choice([0.0, 0.2]), x=x, w=rng.choice([x, x, "f32"]))
    if kind == "weights":
        case["kept"] = rng.choice(["x", "e4m3"])
    return case


# ---------------------------------------------------------------------------
# what a user's program has in hand
# ---------------------------------------------------------------------------
def _tokens(gen, rows, c, dtype):
    """Activations with log-normal channel scales."""
    scale = torch.exp(torch.randn(c, generator=gen, device=DEV))
    return (torch.randn((rows, c), generator=gen, device=DEV) * scale).to(dtype)


def _segments(case, seed):
    """Where the segments begin (skewed lengths, empty ones among them), and whose adapter each takes."""
    rng = np.random.default_rng(seed)
    n = case["segments"]
    share = rng.dirichlet(np.full(n, 0.7))
    offsets = np.concatenate([[0], np.cumsum(rng.multinomial(case["rows"], share / share.sum()))]).astype(np.int64)
    if n == case["adapters"] and case["bare"] == 0.0:
        ids = np.arange(n)  # sorted by adapter, as training has them
    else:
        ids = np.minimum(rng.zipf(1.5, n) - 1, rng.integers(0, case["adapters"], n))
        ids[rng.random(n) < case["bare"]] = -1
    if case["single"]:
        offsets = np.arange(n + 1, dtype=np.int64)
    return offsets, ids.astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    kind, dt = case["kind"], _dtype(case["x"])
    st = dict(case=case)
    rows, c_in = case["rows"], case["c_in"]
    if kind in ("pack", "unpack"):
        st["x"] = _tokens(gen, rows, c_in, dt)
        if kind == "unpack":
            st["values"], st["scales"] = _packed(st.pop("x"))
        return st
    c_out, rank, n, wt = case["c_out"], case["rank"], case["adapters"], _dtype(case["w"])
    offsets, ids = _segments(case, seed)
    st["longest"] = int(np.diff(offsets).max())
    st["whole"] = torch.from_numpy(offsets).to(DEV)
    st["offsets"] = None if case["single"] else st["whole"]
    st["ids"] = torch.from_numpy(ids).to(DEV)
    st["scale"] = 0.5 + torch.rand(n, generator=gen, device=DEV)
    st["a"] = (torch.randn((n, rank, c_in), generator=gen, device=DEV) * c_in ** -0.5).to(wt)
    st["b"] = (torch.randn((n, rank, c_out), generator=gen, device=DEV) * 0.05).to(wt)
    if kind != "grad":
        st["x"] = _tokens(gen, rows, c_in, dt)
    if kind != "lora":
        st["dy"] = _tokens(gen, rows, c_out, dt)
    if kind != "weights":
        st["base"] = torch.randn((rows, c_out if kind == "lora" else c_in), generator=gen, device=DEV).to(dt)
        return st
    # what the passes before left: the rows in the adapters' ranks, both ways
    st["s"], _ = _through(st, st["x"], st["a"], None)
    st["ds"], _ = _through(st, st["dy"], st["b"], None)
    if case["kept"] == "e4m3":
        st["x"], st["scales"] = _packed(st["x"])
    del st["a"], st["b"]
    return st


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits
# ---------------------------------------------------------------------------
def _places(st):
    """For every (segment, place): its row (one past the last where there is none)."""
    rows = st["case"]["rows"]
    at = st["whole"][:-1, None] + torch.arange(st["longest"], device=DEV)
    return torch.where(at < st["whole"][1:, None], at, torch.full_like(at, rows))


def _by_segment(x, at):
    x = x.float()
    return torch.cat([x, x.new_zeros((1, x.shape[1]))])[at]


def _of_adapter(st, m):
    """Each segment's adapter (zeros for none)."""
    ids = st["ids"].long()
    live = (ids >= 0) & (ids < m.shape[0])
    return torch.where(live.view(-1, *[1] * (m.dim() - 1)), m.float()[ids.clamp(min=0)], 0.0)


def _through(st, x, inner, outer):
    """(x inner^T, scale (x inner^T) outer), each row with its own segment's adapter."""
    rows, at = st["case"]["rows"], _places(st)
    s = torch.bmm(_by_segment(x, at), _of_adapter(st, inner).transpose(1, 2).contiguous())

    def back(v):
        out = v.new_empty((rows + 1, v.shape[2]))
        out[at.reshape(-1)] = v.flatten(0, 1)
        return out[:rows].clone()

    if outer is None:
        return back(s), None
    d = torch.bmm(s, _of_adapter(st, outer)) * _of_adapter(st, st["scale"]).view(-1, 1, 1)
    return back(s), back(d)


def _shared_power(most):
    """The exponent of the smallest power of two p with most <= 448 p, at least -127."""
    m, e = torch.frexp(most)
    return torch.where(most > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127)


def _packed(x):
    rows, c = x.shape
    blocks = -(-c // SHARED)
    b = torch.nn.functional.pad(x.float(), (0, blocks * SHARED - c)).view(rows, blocks, SHARED)
    e = _shared_power(b.abs().amax(dim=-1))
    v = torch.ldexp(torch.ldexp(b, (-e).div(2, rounding_mode="floor").unsqueeze(-1)), (-e - (-e).div(2, rounding_mode="floor")).unsqueeze(-1))
    values = v.flatten(1)[:, :c].to(torch.float8_e4m3fn).contiguous()
    return values.view(torch.uint8), (e + 127).to(torch.uint8)


def _unpacked(values, scales):
    v = values.view(torch.float8_e4m3fn).float()
    p = torch.exp2(scales.double() - 127).float()
    return v * p.repeat_interleave(SHARED, dim=1)[:, :v.shape[1]]


def _plain(st):
    case = st["case"]
    kind, dt = case["kind"], _dtype(case["x"])
    if kind == "pack":
        values, scales = _packed(st["x"])
        return dict(values=values.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))
    if kind == "unpack":
        return _unpacked(st["values"], st["scales"]).to(dt)
    if kind == "lora":
        return (st["base"].float() + _through(st, st["x"], st["a"], st["b"])[1]).to(dt)
    if kind == "grad":
        return (st["base"].float() + _through(st, st["dy"], st["b"], st["a"])[1]).to(dt)
    at = _places(st)
    ids = st["ids"].long()
    mine = (ids == torch.arange(case["adapters"], device=DEV).unsqueeze(1)).float() * st["scale"].unsqueeze(1)
    x = _unpacked(st["x"], st["scales"]) if case["kept"] == "e4m3" else st["x"]

    def grad(p, x):
        part = torch.bmm(_by_segment(p, at).transpose(1, 2).contiguous(), _by_segment(x, at))
        return (mine @ part.flatten(1)).view(-1, *part.shape[1:])

    return dict(da=grad(st["ds"], x), db=grad(st["s"], st["dy"]))


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _framework(st):
    import nvfp4_scale_calibration_amd as lh

    case = st["case"]
    kind, dt = case["kind"], _dtype(case["x"])
    if kind == "pack":
        values, scales = lh.lh_checkpoint_pack(st["x"])
        return dict(values=values.view(torch.float8_e4m3fn), scales=scales.view(torch.float8_e8m0fnu))
    if kind == "unpack":
        return lh.lh_checkpoint_unpack(st["values"], st["scales"], out_dtype=dt)
    if kind == "lora":
        return lh.lh_lora(st["x"], st["a"], st["b"], st["scale"], offsets=st["offsets"], adapter_ids=st["ids"], base=st["base"])
    if kind == "grad":
        return lh.lh_lora_grad(st["dy"], st["a"], st["b"], st["scale"], offsets=st["offsets"], adapter_ids=st["ids"], base=st["base"])
    da, db = lh.lh_lora_weight_grad(st["x"], st["dy"], st["s"], st["ds"], case["adapters"], st["scale"], offsets=st["offsets"],
                                    adapter_ids=st["ids"], x_scale=st.get("scales"))
    return dict(da=da, db=db)


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    e = 2 if case["x"] == "bf16" else 4
    kind, t, c = case["kind"], case["rows"], case["c_in"]
    if kind in ("pack", "unpack"):
        return dict(bytes=t * c * (e + 1) + t * -(-c // SHARED), flops=2 * t * c)
    o, r = case["c_out"], case["rank"]
    used = min(case["adapters"], case["segments"])
    flops = 2 * t * r * (c + o)
    if kind == "weights":
        kept = t * c + t * -(-c // SHARED) if case["kept"] == "e4m3" else t * c * e
        return dict(bytes=kept + t * o * e + 2 * t * r * 4 + case["adapters"] * r * (c + o) * 4, flops=flops)
    ew = 2 if case["w"] == "bf16" else 4
    rest = t * (c + 2 * o) if kind == "lora" else t * (o + 2 * c)
    return dict(bytes=rest * e + used * r * (c + o) * ew, flops=flops)


def _decoded64(values, scales, cols):
    """A checkpoint by its formats' bit fields: sign, exponent and mantissa of E4M3, the shared exponent."""
    v = values.double()
    sign = torch.where(v >= 128, -1.0, 1.0)
    m = torch.remainder(v, 128)
    ex, man = torch.floor(m / 8), torch.remainder(m, 8)
    mag = torch.where(ex == 0, man * 2.0 ** -9, torch.exp2(ex - 7) * (1 + man / 8))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(SHARED, dim=1)[:, :cols]


def exact(case, seed):
    kind = case["kind"]
    st = prepare(case, seed)
    if kind == "unpack":
        rows = st["values"].shape[0]
        slab = max(1, (1 << 25) // case["c_in"])
        got = torch.empty((rows, case["c_in"]), dtype=torch.float64, device=DEV)
        for r0 in range(0, rows, slab):
            got[r0:r0 + slab] = _decoded64(st["values"][r0:r0 + slab], st["scales"][r0:r0 + slab], case["c_in"])
        return got
    if kind == "pack":
        # the values are by definition the points of the E4M3 grid nearest to the quotients, ties to the even code
        x = st["x"]
        rows, c = x.shape
        codes = torch.arange(127, dtype=torch.uint8, device=DEV).view(1, -1)
        grid = _decoded64(codes, torch.full((1, 4), 127, dtype=torch.uint8, device=DEV), 127)[0]
        mid = (grid[1:] + grid[:-1]) / 2
        powers = torch.exp2(torch.arange(-127, 128, device=DEV).double())
        blocks = -(-c // SHARED)
        values = torch.empty((rows, c), dtype=torch.float64, device=DEV)
        scales = torch.empty((rows, blocks), dtype=torch.float64, device=DEV)
        slab = max(1, (1 << 24) // c)
        for r0 in range(0, rows, slab):
            part = x[r0:r0 + slab].double()
            b = torch.zeros((part.shape[0], blocks * SHARED), dtype=torch.float64, device=DEV)
            b[:, :c] = part
            b = b.view(-1, blocks, SHARED)
            p = powers[torch.bucketize(b.abs().amax(dim=-1), 448 * powers, right=False)]
            q = (b / p.unsqueeze(-1)).flatten(1)[:, :c].contiguous()
            lo, hi = torch.bucketize(q.abs(), mid, right=False), torch.bucketize(q.abs(), mid, right=True)
            k = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
            values[r0:r0 + slab] = grid[k] * torch.sign(q)
            scales[r0:r0 + slab] = p
        return dict(values=values, scales=scales)
    offsets, ids, scale = st["whole"].tolist(), st["ids"].tolist(), st["scale"].tolist()
    n = case["adapters"]
    if kind == "weights":
        x = _decoded64(st["x"], st["scales"], case["c_in"]) if case["kept"] == "e4m3" else st["x"]
        da = torch.zeros((n, case["rank"], case["c_in"]), dtype=torch.float64, device=DEV)
        db = torch.zeros((n, case["rank"], case["c_out"]), dtype=torch.float64, device=DEV)
        for i, g in enumerate(ids):
            rows = slice(offsets[i], offsets[i + 1])
            if 0 <= g < n and offsets[i + 1] > offsets[i]:
                da[g] += scale[g] * torch.mm(st["ds"][rows].double().t(), x[rows].double())
                db[g] += scale[g] * torch.mm(st["s"][rows].double().t(), st["dy"][rows].double())
        return dict(da=da, db=db)
    x, inner, outer = (st["x"], st["a"], st["b"]) if kind == "lora" else (st["dy"], st["b"], st["a"])
    y = st["base"].double()
    for i, g in enumerate(ids):
        rows = slice(offsets[i], offsets[i + 1])
        if 0 <= g < n and offsets[i + 1] > offsets[i]:
            y[rows] += scale[g] * torch.mm(torch.mm(x[rows].double(), inner[g].double().t()), outer[g].double())
    return y
