"""64-bit plain forms of the prompt-side operators of the paged cache, and
the tolerances their kernels are held to."""
import math

import torch


def attention(q, k, v, first):
    """One sequence: q [n,Hq,D] at positions first .., k, v [m,Hkv,D] at
    0 .. m-1 (any dtype).  Returns out [n,Hq,D], spread = sum_j p_j |v_j|
    (what a relative error of the weights can move), lse [n,Hq] and the
    largest sum_d |q_d k_d| * scale over the visible pairs, all in 64 bits.
    Invisible keys take no part, whatever they hold."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    out = torch.zeros((n, Hq, D), dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    lse = torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    mag = 0.0
    pos = first + torch.arange(n, device=q.device)
    seen = torch.arange(m, device=q.device)[None] <= pos[:, None]
    for h in range(Hq):
        kk, vv, qq = k[:, h // G].double(), v[:, h // G].double(), q[:, h].double()
        s = (qq @ kk.nan_to_num(0.0, 0.0, 0.0).T) / math.sqrt(D)
        bad = torch.isnan(kk).any(1)  # a NaN key is NaN for the rows that see it
        s = torch.where(bad[None], math.nan, s).masked_fill(~seen, -math.inf)
        mag = max(mag, float(((qq.abs() @ kk.nan_to_num(0.0, 0.0, 0.0).abs().T) / math.sqrt(D)).max()) if m and n else 0.0)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        nonfin = ~torch.isfinite(vv)
        clean = torch.where(nonfin, 0.0, vv)
        out[:, h] = p @ clean
        if bool(nonfin.any()):  # a non-finite V element reaches exactly the rows that see it
            for j, d in nonfin.nonzero().tolist():
                out[seen[:, j], h, d] += vv[j, d]
        spread[:, h] = p @ clean.abs()
        lse[:, h] = z
    return out, spread, lse, mag


def tolerances(dtype, D, spread, out, lse, mag):
    """Elementwise bounds on |out - exact| and |lse - exact|.

    A score is a sum of D fp32-accumulated products: off by at most
    ds = D 2^-24 mag, plus the scaling and the subtraction of the maximum (two
    roundings of values up to 2 mag, taken as 4 mag 2^-24).  A weight is then
    off by ds relative, plus the exponential (2^-12 in the bf16 kernels, whose
    weights are rounded to bf16 anyway; 2^-21 in fp32), in numerator and
    denominator.  bf16 weights are rounded by 2^-8 relative each and the
    output by 2^-8 of itself; fp32 sums over the keys add 2^-20 (running sums
    of at most 2^12 partial sums per accumulator, errors of one sign unlikely)."""
    ds = (D + 4) * 2.0 ** -24 * mag
    if dtype == torch.bfloat16:
        w = 2 * (ds + 2.0 ** -12)
        return (2.0 ** -8 + w) * spread + 2.0 ** -8 * out.abs() + 1e-6, ds + 2.0 ** -12 + 2.0 ** -20 * (1 + lse.abs())
    w = 2 * (ds + 2.0 ** -20)
    return w * spread + 2.0 ** -24 * out.abs() + 1e-7, ds + 2.0 ** -20 * (1 + lse.abs())


def check(got, got_lse, dtype, D, ref, what=""):
    """The output and lse of one sequence against ``attention``'s."""
    out, spread, lse, mag = ref
    to, tl = tolerances(dtype, D, spread, torch.nan_to_num(out, 0.0, 0.0, 0.0), lse, mag)
    g = got.double()
    fin = torch.isfinite(out)
    assert torch.equal(torch.isfinite(g), fin), f"{what}: finite values where the reference has none, or the reverse"
    assert torch.equal(torch.isnan(g), torch.isnan(out)), f"{what}: NaN in other places"
    err = torch.where(fin, g - torch.where(fin, out, 0.0), 0.0).abs()
    over = err > to
    assert not bool(over.any()), (f"{what}: {int(over.sum())} of {over.numel()} off, worst {float((err - to).max()):.3g} "
                                  f"over its bound at {over.nonzero()[0].tolist()}")
    if got_lse is not None:
        fin = torch.isfinite(lse)
        assert torch.equal(torch.isfinite(got_lse), fin), f"{what}: lse"
        e = torch.where(fin, got_lse.double() - torch.where(fin, lse, 0.0), 0.0).abs()
        assert bool((e <= torch.where(fin, tl, 0.0)).all()), f"{what}: lse off by {float(e.max()):.3g}"


def plan(prefix, new, owned, table, free, room, page_size, max_tokens):
    """kv_page_plan on Python lists, one sequence after the other.  ``free``:
    the stack (top last).  Returns (row_start, slots, owned, table, stack,
    refused)."""
    B, max_pages = len(prefix), len(table[0])
    table = [list(r) for r in table]
    stack, owned = list(free), list(owned)
    for b in range(B):
        if new[b] == -1:
            stack += table[b][:owned[b]]
    need = []
    for b in range(B):
        want = -(-(prefix[b] + max(new[b], 0) + room) // page_size)
        need.append(0 if new[b] < 0 or want > max_pages else max(0, want - owned[b]))
    refused, taken = set(), 0
    avail = len(stack)
    for b in range(B):
        taken += need[b]
        want = -(-(prefix[b] + max(new[b], 0) + room) // page_size)
        if new[b] >= 0 and (want > max_pages or (need[b] and taken > avail)):
            refused.add(b)
    full = list(stack)
    popped = 0
    for b in range(B):
        start = sum(need[:b])
        if b in refused or new[b] < 0:
            continue
        for i in range(need[b]):
            table[b][owned[b] + i] = full[avail - 1 - (start + i)]
        owned[b] += need[b]
        popped += need[b]
    row, slots = [0], []
    for b in range(B):
        n = max(new[b], 0)
        row.append(row[-1] + n)
        for i in range(n):
            pos = prefix[b] + i
            slots.append(-1 if b in refused else table[b][pos // page_size] * page_size + pos % page_size)
        if new[b] == -1:
            owned[b] = 0
    slots += [-1] * (max_tokens - len(slots))
    return row, slots, owned, table, full, avail - popped, refused
