"""The router's balance on the GPU against 64-bit references: choice, weights, counts, loss and gradients."""

import pytest
import torch

import lru_expert_cache_amd as ft
from tests import around_case as ac

pytestmark = pytest.mark.gpu

# (tokens, experts, top_k, row padding)
SIZES = [(4, 512, 16, 0), (5, 400, 3, 0), (32, 512, 9, 1), (1, 1, 1, 0), (1, 8, 2, 0), (3, 5, 5, 1), (2, 64, 8, 0), (17, 65, 4, 3), (64, 16, 2, 0), (100, 60, 6, 0), (255, 128, 8, 0),
         (509, 128, 8, 64), (33, 129, 1, 0), (77, 160, 8, 0), (40, 256, 16, 0), (90, 257, 3, 0), (31, 300, 16, 5), (50, 512, 8, 0),
         (5000, 128, 8, 0), (9001, 256, 6, 0)]


@pytest.mark.parametrize("type_", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES)
def test_step(size, type_):
    b = ac.Balance(*size[:3], type_, pad=size[3])
    f, r = b.forward(), b.reference()
    assert torch.equal(f["sel"], r["sel"]) and torch.equal(f["counts"], r["counts"])
    ac.check(f["w"], r["w"], "w")
    ac.check(f["loss"], r["loss"], "loss")
    for dw, dloss in ((True, True), (False, True), (True, False)):
        ac.check(b.backward(f, dw, dloss), b.backward_reference(dw, dloss), f"dlogits {dw} {dloss}")
    f2 = b.forward()
    assert all(torch.equal(f[k], f2[k]) for k in f)


@pytest.mark.parametrize("experts", [8, 64, 128, 256, 500])
def test_ties_go_to_the_lowest_index(experts):
    b = ac.Balance(200, experts, min(8, experts), ties=True)
    b.z[0] = 0.0
    b.z[1, ::2] = -0.0
    b.z[1, 1::2] = 0.0
    b.z[2] = torch.finfo(torch.float32).min
    f, r = b.forward(), b.reference()
    assert torch.equal(f["sel"], r["sel"]) and torch.equal(f["counts"], r["counts"])
    ac.check(f["w"], r["w"], "w")
    ac.check(b.backward(f), b.backward_reference(), "dlogits")


def test_masked_experts_and_tokens():
    """Logits of -inf are never chosen; rows of nothing else, and rows that are masked, count for nothing, whatever they hold."""
    for experts, k in ((6, 4), (130, 16)):
        b = ac.Balance(60, experts, k)
        b.valid = torch.ones(60, dtype=torch.bool, device="cuda")
        b.z[:, 1] = float("-inf")
        b.z[3] = float("-inf")
        b.z[4] = float("-inf")
        b.z[4, 2] = 1.0  # one expert left
        b.z[5, 3:] = float("-inf")  # two of them
        f, r = b.forward(), b.reference()
        assert torch.equal(f["sel"], r["sel"]) and torch.equal(f["counts"], r["counts"])
        assert f["sel"][4].tolist() == [2] + [-1] * (k - 1) and f["w"][4].tolist() == [1.0] + [0.0] * (k - 1)
        ac.check(f["w"], r["w"], "w")
        ac.check(f["loss"], r["loss"], "loss")
        dz = b.backward(f)
        ac.check(dz, b.backward_reference(), "dlogits")
        assert (dz[3] == 0).all() and (dz[:, 1] == 0).all()
        # what a masked row holds is not seen
        b.valid[7:11] = False
        f, dz = b.forward(), b.backward(b.forward())
        b.z[7], b.z[8], b.z[9] = float("nan"), float("inf"), float("-inf")
        f2, dz2 = b.forward(), b.backward(b.forward())
        assert all(torch.equal(f[n], f2[n]) for n in f) and torch.equal(dz, dz2)
        assert (f["sel"][7:11] == -1).all() and (f["w"][7:11] == 0).all() and (dz[7:11] == 0).all()


def test_nothing_counts():
    b = ac.Balance(30, 20, 4)
    b.valid = torch.zeros(30, dtype=torch.bool, device="cuda")
    f = b.forward()
    assert f["loss"] == 0 and (f["counts"] == 0).all() and (f["sel"] == -1).all()
    assert (b.backward(f) == 0).all()
    b = ac.Balance(0, 20, 4)
    f = b.forward()
    assert f["loss"] == 0 and (f["counts"] == 0).all()
    b.backward(f)


def test_nan_and_infinity_stay_in_their_token():
    b = ac.Balance(40, 100, 8, masked=0)
    b.z[3, 50], b.z[9, 2] = float("nan"), float("inf")
    f = b.forward()
    assert torch.isnan(f["loss"]).all() and not (f["sel"][3] == 50).any() and f["sel"][9, 0] == 2
    assert len(set(f["sel"][3].tolist())) == 8
    dz = b.backward(f)
    bad = torch.isnan(dz).any(1)
    assert bad[3] and bad[9] and int(bad.sum()) == 2


def test_same_choice_as_the_layers_router():
    """Choice and weights as the routed layer makes them of the same logits (with ties among them)."""
    from oracle import router

    b = ac.Balance(64, 16, 2, masked=0, ties=True)
    f = b.forward()
    z = b.z.double().cpu().numpy()
    sel = router.select_topk(z, 2)
    assert (f["sel"].cpu().numpy() == sel).all()
    assert abs(f["w"].cpu().numpy() - router.topk_weights(z, sel)).max() < 1e-6


def test_loss_of_equal_experts_is_the_weight():
    """Uniform probabilities, choices spread evenly: the loss is `weight`."""
    b = ac.Balance(64, 64, 1, weight=0.25, masked=0)
    b.z.copy_(torch.eye(64, device="cuda") * 1e-6)
    f = b.forward()
    assert (f["counts"][:64] == 1).all() and abs(float(f["loss"]) - 0.25) < 0.25 * 2e-6


def test_gradients_follow_differences():
    """The counts held, the loss and the weights differentiated along a random direction."""
    b = ac.Balance(12, 20, 4, masked=0.2, weight=3.0)
    f, dz = b.forward(), b.backward(b.forward())
    ref = b.backward_reference()
    z, p, ep, w, ew, c, sel, some, on = b.dref

    def total(z):
        q = torch.softmax(z, 1) * on[:, None]
        v = torch.softmax(torch.gather(z, 1, sel), 1) * on[:, None]
        return float(b.dloss) * (q.sum(0) * c).sum() + (v * b.dw.double()).sum()

    v = torch.randn(z.shape, generator=ac.gen(4), device="cuda", dtype=torch.float64)
    step = 2.0**-14
    difference = (total(z + step * v) - total(z - step * v)) / (2 * step)
    # the third derivative of a softmax along v is a few times |v|^3 its value: 2^-28 / 6 of that
    bound = (ref[1] * v.abs()).sum() + 1e-7 * (v.abs() ** 3).sum()
    assert (difference - (dz.double() * v).sum()).abs() <= bound


def test_counts_of_several_ranks():
    """Two halves of a batch, their counts added: the gradients of the whole batch's loss."""
    whole = ac.Balance(90, 40, 4, masked=0.1)
    f = whole.forward()
    dz = whole.backward(f)
    for lo, hi in ((0, 37), (37, 90)):
        d = ft.make_balance(ft.FT_DT_F32, hi - lo, 40, 4, whole.weight)
        out = torch.empty(hi - lo, 40, device="cuda")
        ft.ft_moe_balance_backward(d, whole.z[lo:hi], whole.valid[lo:hi], f["sel"][lo:hi], f["w"][lo:hi], f["counts"],
                                   whole.dw[lo:hi], whole.dloss, out)
        assert torch.equal(out, dz[lo:hi])


def test_an_expert_given_twice_counts_twice():
    b = ac.Balance(5, 30, 3, masked=0)
    f = b.forward()
    once = b.backward(f, dloss=False)
    f["sel"][2, 1] = f["sel"][2, 0]
    dz = b.backward(f, dloss=False)
    w, v = f["w"][2].double(), b.dw[2].double()
    one = w * (v - (w * v).sum())
    got = dz.double()[2, int(f["sel"][2, 0])]
    base = b.backward(f, dw=False, dloss=False).double()[2, int(f["sel"][2, 0])]
    # sums of three numbers of this size, a few roundings each
    assert abs(got - base - one[0] - one[1]) < 16 * ac.E * (w * v.abs()).sum() + 4 * ac.E * abs(base)
    keep = torch.arange(5, device="cuda") != 2
    assert torch.equal(dz[keep], once[keep])


def test_in_place():
    b = ac.Balance(50, 100, 4, pad=4)
    f = b.forward()
    dz = b.backward(f)
    ft.ft_moe_balance_backward(b.d, b.z, b.valid, f["sel"], f["w"], f["counts"], b.dw, b.dloss, b.z)
    assert torch.equal(b.z, dz)


def test_rows_beyond_4_gb():
    """Offsets of more than 32 bits: rows far apart."""
    b = ac.Balance(40, 100, 4)
    f = b.forward()
    dz, ld = b.backward(f), 1 << 25
    assert 39 * ld * 4 > 2**32
    b.z = torch.as_strided(torch.empty(39 * ld + 100, device="cuda"), (40, 100), (ld, 1)).copy_(b.z)
    b.d.ld_logits = ld
    f2 = b.forward()
    assert all(torch.equal(f[k], f2[k]) for k in f)
    ft.ft_moe_balance_backward(b.d, b.z, b.valid, f["sel"], f["w"], f["counts"], b.dw, b.dloss, b.z)
    assert torch.equal(b.z, dz)


@pytest.mark.parametrize("experts,k", [(2, 2), (8, 8), (16, 16), (130, 16), (250, 16), (500, 16)])
def test_probabilities_keep_their_bits_at_any_distance(experts, k):
    """Logits up to 110 below the largest, at differences that 32 bits hold: the bounds do not grow with the distance,
    and reach into the subnormal numbers."""
    T, tiny = 300, 2.0**-149
    b = ac.Balance(T, experts, k, masked=0)
    b.z.copy_((torch.rand(T, experts, generator=ac.gen(6), device="cuda") * -880).round() / 8)
    at = torch.arange(T, device="cuda")
    b.z[at, at % experts] = 0.0
    f, r = b.forward(), b.reference()
    assert torch.equal(f["sel"], r["sel"]) and torch.equal(f["counts"], r["counts"])
    _, p, _, w, _, c, _, _, _ = b.dref
    # an exponential is off by 3 E: its argument, at most ln 2 / 2, by less than one (two roundings of half a unit and
    # the product with log2 e), exp2 by a unit.  The sum carries that and rounds for each term: w's 6 steps between lanes,
    # p's 7 within a lane too.  The quotient rounds once.
    ac.check(f["w"], (w, 14 * ac.E * w + tiny), "w")
    ep = 21 * ac.E * p + tiny
    loss = (c * p.sum(0)).sum()
    ac.check(f["loss"], (loss[None], ((c * (ep.sum(0) + (T / 64 + 24) * ac.E * p.sum(0))).sum() + 2 * ac.E * loss)[None]), "loss")
    s = (p * c).sum(1, keepdim=True)
    dz, es = p * (c - s), (ep * c).sum(1, keepdim=True) + 20 * ac.E * s
    ac.check(b.backward(f, dw=False, dloss=False), (dz, ep * (c - s).abs() + p * (3 * ac.E * c + es) + 4 * ac.E * dz.abs() + tiny), "dlogits")
