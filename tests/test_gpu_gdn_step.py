"""Gated delta steps (moe_gdn_step) against their plain binary64 form.

Tolerances: the state is binary32 and a step is a contraction for these inputs (decay <= 1, unit
keys, write strength in (0, 1)); a row takes two dots of 128 terms and three more operations, so
one step is off by less than 2 * 128 * 2^-24 * max(1, |S|) = 1.6e-5 in the worst case; outputs
add one rounding to bf16, 2^-8 relative."""

import numpy as np
import pytest

from gpu_helpers import ensure_lib, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_lib()


def _inputs(slot, n_slots, hk, hv, seed):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    R = len(slot)

    def unit():
        x = torch.randn((R, hk, 128), generator=g, device="cuda")
        return (x / x.norm(dim=-1, keepdim=True)).bfloat16()

    return dict(q=unit(), k=unit(), v=torch.randn((R, hv, 128), generator=g, device="cuda").bfloat16(),
                alpha=torch.rand((R, hv), generator=g, device="cuda"), beta=torch.rand((R, hv), generator=g, device="cuda"),
                state=torch.randn((n_slots, hv, 128, 128), generator=g, device="cuda"),
                slot=torch.tensor(slot, dtype=torch.int32, device="cuda"))


def _check(d, what, steps=1):
    from oracle import serve
    from sparse_moe_02_amd.gdn import gdn_step

    ref = {k: v.double().cpu().numpy() for k, v in d.items() if k != "slot"}
    slot = d["slot"].cpu().numpy()
    ro, rS = serve.gdn_step(ref["q"], ref["k"], ref["v"], ref["alpha"], ref["beta"], ref["state"], slot)
    out = gdn_step(**d).double().cpu().numpy()
    S = d["state"].double().cpu().numpy()
    tol = steps * 1.6e-5 * max(1.0, np.abs(rS).max())
    say(f"{what}: state error {np.abs(S - rS).max():.3g} (limit {tol:.3g})")
    assert (np.abs(S - rS) <= tol).all()
    assert (np.abs(out - ro) <= 2.0 ** -8 * np.abs(ro) + 12 * tol).all()  # |q|_1 <= sqrt(128) < 12
    named = {int(s) for s in slot if 0 <= s < S.shape[0]}
    for s in set(range(S.shape[0])) - named:
        assert np.array_equal(S[s], ref["state"][s])  # slots that no row names keep their bits
    for r, s in enumerate(slot):
        if not 0 <= s < S.shape[0]:
            assert (out[r] == 0).all()


@pytest.mark.parametrize("hk,hv", [(16, 32), (1, 1), (3, 3), (2, 8)])
@pytest.mark.parametrize("R", [1, 2, 5])
def test_one_row_per_slot(R, hk, hv):
    _check(_inputs(list(np.random.default_rng(R).permutation(R + 2)[:R]), R + 2, hk, hv, R), f"{R} rows, {hk}/{hv}")


def test_rows_of_one_slot_in_order():
    _check(_inputs([3, 0, 3, 3, 1, 0, 3], 5, 2, 4, 7), "repeated slots", 4)


def test_many_rows_of_few_slots():
    """More rows than a workgroup has threads; one slot's rows far apart."""
    slot = [i % 2 for i in range(300)] + [2] * 5 + [0]
    _check(_inputs(slot, 3, 1, 1, 8), "300 rows", 151)


def test_padding_rows():
    _check(_inputs([-1, 1, 4, 2 ** 31 - 1, 0, -2 ** 31], 4, 2, 4, 9), "padding")


def test_all_rows_padding():
    _check(_inputs([-1, -1], 2, 2, 2, 10), "all padding")


def test_extreme_gates():
    d = _inputs([0, 1, 2, 3], 4, 2, 4, 11)
    d["alpha"][0] = 0.0
    d["alpha"][1] = 1.0
    d["beta"][2] = 0.0
    d["beta"][3] = 1.0
    d["alpha"][3, 0] = 1e-38
    _check(d, "extreme gates")


def test_a_decay_of_zero_starts_anew_whatever_the_slot_held():
    import torch

    from sparse_moe_02_amd.gdn import gdn_step

    d = _inputs([0, 1, 1, 2], 4, 2, 4, 15)
    d["alpha"][0] = 0.0  # the slot's first row
    d["alpha"][2, 1] = 0.0  # its second row, one head
    clean = {k: v.clone() for k, v in d.items()}
    clean["state"][0] = 0.0
    d["state"][0] = float("nan")
    d["state"][0, 1] = float("inf")
    out, ref = gdn_step(**d), gdn_step(**clean)
    assert torch.equal(out, ref) and torch.equal(d["state"], clean["state"])
    _check({**_inputs([0, 1, 1, 2], 4, 2, 4, 15), "alpha": d["alpha"].clone()}, "decays of zero")


def test_steps_follow_the_scan():
    """A prompt's scan, then its next tokens as steps: the scan over all of them."""
    import torch

    from sparse_moe_02_amd.gdn import gdn_scan, gdn_step

    d = _inputs([0] * 40, 1, 2, 4, 12)
    d.pop("slot")
    d["alpha"] = 0.9 + 0.1 * d["alpha"]
    whole = {k: v.clone() for k, v in d.items()}
    ro = gdn_scan(whole["q"], whole["k"], whole["v"], whole["alpha"], whole["beta"], whole["state"][0])
    pool = torch.zeros((3, 4, 128, 128), device="cuda")
    pool[2] = d["state"][0]
    part = {k: v[:33] for k, v in d.items() if k != "state"}
    outs = [gdn_scan(*(part[k] for k in ("q", "k", "v", "alpha", "beta")), pool[2])]
    for t in range(33, 40):
        outs.append(gdn_step(*(d[k][t:t + 1] for k in ("q", "k", "v", "alpha", "beta")), pool,
                             torch.tensor([2], dtype=torch.int32, device="cuda")))
    out = torch.cat(outs)
    S, rS = pool[2].double(), whole["state"][0].double()
    assert (S - rS).abs().max() <= 40 * 1.6e-5 * max(1.0, float(rS.abs().max()))
    assert ((out.double() - ro.double()).abs() <= 2.0 ** -7 * ro.double().abs() + 40 * 12 * 1.6e-5).all()
    assert (pool[:2] == 0).all()


def test_state_beyond_32_bits():
    """A pool of more than 2^31 elements: the last slot."""
    import torch

    from sparse_moe_02_amd.gdn import gdn_step

    n = 2 ** 31 // (32 * 128 * 128) + 2
    d = _inputs([0], 1, 16, 32, 13)
    big = torch.empty((n, 32, 128, 128), device="cuda")
    big[-1] = d["state"][0]
    out = gdn_step(**{**d, "state": big, "slot": torch.tensor([n - 1], dtype=torch.int32, device="cuda")})
    ref = gdn_step(**d)
    assert (out == ref).all() and (big[-1] == d["state"][0]).all()


def test_graph_replays_read_the_slots():
    import torch

    from sparse_moe_02_amd.gdn import gdn_step

    d = _inputs([0, 1, 2], 6, 2, 4, 14)
    e = {k: v.clone() for k, v in d.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = gdn_step(**d)
    for i in range(4):
        slot = torch.tensor([i, 5, (3 * i) % 5], dtype=torch.int32, device="cuda")
        d["slot"].copy_(slot)
        e["slot"].copy_(slot)
        torch.cuda.synchronize()
        g.replay()
        ref = gdn_step(**e)
        torch.cuda.synchronize()
        assert (out == ref).all() and (d["state"] == e["state"]).all(), i
