"""The norms bit for bit: codes and scales of rows whose norm is exactly 1, and every row written in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import routed_expert_moe_b200 as m
    return m


def unit_rows(T, H, seed):
    """[T, H] multiples of 1/8 whose squares add up to H, exactly in fp32 and in any order: a root of the mean of 1."""
    g = torch.Generator().manual_seed(seed)
    n = (torch.randn(T, H, generator=g) * 8).round().long().clamp(-60, 60)
    for t in range(T):
        row, order = n[t], torch.randperm(H, generator=g).tolist()
        gap = 64 * H - int((row * row).sum())
        for i in order:                      # towards the target, a value at a time
            step = 1 if gap > 0 else -1
            a = int(row[i].abs())
            d = (a + step) ** 2 - a * a
            if 1 < a < 60 and abs(gap) >= abs(d):
                row[i] = (a + step) * (1 if row[i] > 0 else -1)
                gap -= d
        for i in order:                      # what is left over, in ones
            a = int(row[i])
            if gap > 0 and a == 0:
                row[i], gap = 1, gap - 1
            elif gap < 0 and abs(a) == 1:
                row[i], gap = 0, gap + 1
        assert gap == 0
    return (n.float() / 8).to(torch.bfloat16)


def formula(v, H):
    """codes = e4m3(fl32(v * fl32(1 / s))), s = fl32(max|v| / 448), in torch's fp32 on the CPU."""
    kb = (H + 127) // 128
    b = torch.nn.functional.pad(v, (0, kb * 128 - H)).view(-1, kb, 128)
    amax = b.abs().amax(-1)
    s = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    q = b * (torch.ones_like(s) / s)[..., None]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1, kb * 128), s


@pytest.mark.parametrize("T,H", [(1, 256), (7, 2688), (450, 272), (450, 2704), (460, 4112), (3, 8208), (450, 8208)])
def test_codes_are_the_formulas(moe, T, H):
    rows = unit_rows(min(T, 9), H, seed=H + T)
    x = rows[torch.arange(T) % len(rows)]
    gain = (1 + torch.randn(H, generator=torch.Generator().manual_seed(H)) * 0.3).to(torch.bfloat16)
    v = x.float() * gain.float()             # exact: 8 bits times 8 bits
    want, want_s = formula(v, H)
    kb = want_s.shape[1]
    u = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    codes, scales = torch.empty(T, kb * 128, device="cuda", dtype=torch.uint8), torch.empty(T, kb, device="cuda")
    moe.prenorm(x.cuda(), gain.cuda(), u=u, codes=codes, scales=scales, eps=0.0)
    assert torch.equal(u.cpu(), v.to(torch.bfloat16))
    assert torch.equal(scales.cpu(), want_s)
    assert torch.equal(codes.cpu(), want)
    # a block without output (alpha 0) leaves x, and the norm of it is the same
    x_out = torch.empty_like(u)
    codes.fill_(255)
    moe.postnorm(torch.ones_like(u), None, x.cuda(), x_out, alpha=0.0, eps=0.0, next_gain=gain.cuda(), codes=codes,
                 scales=scales)
    assert torch.equal(x_out.cpu(), x) and torch.equal(codes.cpu(), want) and torch.equal(scales.cpu(), want_s)


@pytest.mark.parametrize("T,H", [(3, 272), (450, 2704), (2, 33040)])
@pytest.mark.parametrize("x_out,u", [("x", None), ("y", None), ("gate", None), (None, "x"), (None, "y"), (None, "gate"),
                                     ("x", "y"), ("y", "x"), ("gate", "x"), ("x", "gate")])
def test_every_row_in_place(moe, T, H, x_out, u):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    t = {k: torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for k in ("x", "y", "gate")}
    gain = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)

    def call(x, y, gate, x_out, u):
        moe.postnorm(y, gain, x, x_out, gate=gate, alpha=0.5, next_gain=gain, u=u)
        return x_out, u

    want = call(**t, x_out=torch.empty_like(t["x"]), u=torch.empty_like(t["x"]))
    c = {k: v.clone() for k, v in t.items()}
    got = call(**c, x_out=c[x_out] if x_out else torch.empty_like(t["x"]), u=c[u] if u else torch.empty_like(t["x"]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for k in c:
        if k not in (x_out, u):
            assert torch.equal(c[k], t[k])
