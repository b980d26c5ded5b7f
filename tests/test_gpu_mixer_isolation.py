"""Packed sequences do not reach one another: with infinities and NaN in one sequence's inputs, what
the calls return for the sequences beside it (outputs, final states, gradients of each token and
of the initial states) is bit for bit what it is without them.  Parameter gradients sum over all
sequences and are left out."""
import pytest
import torch

import chunked_gated_delta_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu

DEV = "cuda"
BAD = [("dy", "inf"), ("dy", "nan"), ("z", "inf"), ("z", "nan"), ("C", "inf"), ("C", "nan"),
       ("dt", "inf"), ("dt", "nan"), ("x", "inf"), ("x", "nan"), ("B", "nan"), ("h0", "nan"),
       ("dht", "inf")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def others(T, cu, bad):
    """Tokens and sequences beside the bad one."""
    tokens = torch.ones(T, dtype=torch.bool, device=DEV)
    tokens[cu[bad]:cu[bad + 1]] = False
    seqs = torch.ones(len(cu) - 1, dtype=torch.bool, device=DEV)
    seqs[bad] = False
    return tokens, seqs


def ssm_inputs(T, n, D, N, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    return dict(x=r(T, D).to(dtype), dt=(r(T, D) * 0.5 - 3).to(dtype), A=-torch.exp(r(D, N) * 0.5),
                B=r(T, 1, N).to(dtype), C=r(T, 1, N).to(dtype), D=r(D), z=r(T, D).to(dtype),
                dt_bias=r(D) * 0.3, h0=r(n, D, N), dy=r(T, D).to(dtype), dht=r(n, D, N))


def ssm_calls(i, cu, backward):
    args = [i[k] for k in ("x", "dt", "A", "B", "C")]
    opts = dict(D=i["D"], z=i["z"], dt_bias=i["dt_bias"], initial_state=i["h0"], cu_seqlens=cu)
    out = dict(zip(("y", "ht"), gdr.ssm_fwd(*args, **opts, output_final_state=True)))
    if backward:
        g = gdr.ssm_bwd(*args, i["dy"], **opts, dfinal_state=i["dht"])
        out.update(dx=g[0], ddt=g[1], dB=g[3], dC=g[4], dz=g[6], dh0=g[8])
    return out


# Bounds inside the ranges of the scans (of 16 to 64 tokens) and on their edges, few and many
# channels; the bad sequence first, in the middle, last, and one of the empty ones' neighbours.
@pytest.mark.parametrize("cu,D,N,bad,at", [
    ([0, 150, 300], 64, 16, 1, 3),
    ([0, 150, 300], 64, 16, 0, 149),
    ([0, 70, 90, 90, 200], 48, 5, 1, 0),
    ([0, 64, 128, 200], 32, 64, 1, 2),
    ([0, 700, 1500], 2048, 16, 1, 1),
    ([0, 410, 450, 1300], 2048, 16, 1, 20),
    ([0, 700, 1000], 1024, 30, 1, 0),
])
@pytest.mark.parametrize("key,value", BAD)
def test_state_space_sequences_beside_a_bad_one(cu, D, N, bad, at, key, value):
    T, n = cu[-1], len(cu) - 1
    i = ssm_inputs(T, n, D, N, torch.bfloat16, T + D)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    clean = ssm_calls(i, cud, True)
    j = {**i, key: i[key].clone()}
    j[key][bad if key in ("h0", "dht") else cu[bad] + at] = float(value)
    tokens, seqs = others(T, cu, bad)
    for k, v in ssm_calls(j, cud, True).items():
        keep = seqs if k in ("ht", "dh0") else tokens
        assert torch.isfinite(clean[k]).all()
        assert torch.equal(v[keep], clean[k][keep]), f"{k} beside {key} = {value}"


@pytest.mark.parametrize("key,value", [b for b in BAD if b[0] not in ("dy", "dht")])
def test_state_space_prompt_with_much_work(key, value):
    cu, D, N, bad = [0, 2100, 2200, 5003], 4096, 16, 1
    i = ssm_inputs(cu[-1], 3, D, N, torch.bfloat16, 1)
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    clean = ssm_calls(i, cud, False)
    j = {**i, key: i[key].clone()}
    j[key][bad if key == "h0" else cu[bad] + 5] = float(value)
    tokens, seqs = others(cu[-1], cu, bad)
    got = ssm_calls(j, cud, False)
    assert torch.equal(got["y"][tokens], clean["y"][tokens])
    assert torch.equal(got["ht"][seqs], clean["ht"][seqs])


@pytest.mark.parametrize("cu,C", [([0, 150, 151, 300], 64), ([0, 1000, 1003, 5003], 6144)])
@pytest.mark.parametrize("key,value", [("x", "inf"), ("x", "nan"), ("dy", "nan"), ("h0", "inf"),
                                       ("dht", "nan")])
def test_convolution_sequences_beside_a_bad_one(cu, C, key, value):
    T, n, bad = cu[-1], len(cu) - 1, 1
    g = torch.Generator(device=DEV).manual_seed(C)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    i = dict(x=r(T, C), dy=r(T, C), h0=r(n, 3, C), dht=r(n, 3, C))
    w, b = r(C, 4).float(), r(C).float()
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)

    def calls(i):
        y, ht = gdr.conv_fwd(i["x"], w, b, i["h0"], cud, "silu", True)
        dx, _, _, dh0 = gdr.conv_bwd(i["x"], w, i["dy"], b, i["h0"], cud, "silu", i["dht"])
        return dict(y=y, ht=ht, dx=dx, dh0=dh0)

    clean = calls(i)
    j = {**i, key: i[key].clone()}
    j[key][bad if key in ("h0", "dht") else cu[bad]] = float(value)
    tokens, seqs = others(T, cu, bad)
    for k, v in calls(j).items():
        keep = seqs if k in ("ht", "dh0") else tokens
        assert torch.equal(v[keep], clean[k][keep]), f"{k} beside {key} = {value}"
