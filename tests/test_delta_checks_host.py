"""The delta rule's checks themselves: mistakes planted in copies of the fp64 model, and taken for a kernel's outputs, are refused by
`delta_helpers.check`; the model's own outputs, rounded once, are not."""
import inspect

import pytest
import torch

import oracle.delta as od
from delta_helpers import DTYPE, FLOAT_OUTPUTS, check, f64, make, reference

DECAY = "            S = S * np.exp(log_a[t])[:, None, None]\n"
ERROR = '            u = beta[t][:, None] * (v[t] - np.einsum("hnp,hn->hp", S, kt))\n'
WRITE = "            S = S + kt[:, :, None] * u[:, None, :]\n"
READ = '            y[t] = scale * np.einsum("hnp,hn->hp", S, qt)\n'
MISTAKES = {  # name: (what stands in the model, what is put there, outputs that it has to show in)
    "decay after the write": (DECAY + ERROR + WRITE, ERROR + WRITE + DECAY, ("y",)),
    "error of the state before its decay": (DECAY + ERROR, ERROR + DECAY, ("y", "final")),
    "no beta on the write": (ERROR, ERROR.replace("beta[t][:, None] * ", ""), ("y", "final")),
    "output before the write": (WRITE + READ, READ + WRITE, ("y",)),
    "dq of the state before the write": ('np.einsum("hnp,hp->hn", S, dy[t])', 'np.einsum("hnp,hp->hn", old, dy[t])', ("dq",)),
    "dk without the error's part": (' - np.einsum("hnp,hp->hn", old, dv[t])', "", ("dk",)),
    "dk without the write's part": ('np.einsum("hnp,hp->hn", dS, beta[t][:, None] * e) - ', "-", ("dk",)),
    "dbeta of the value, not the error": ("(du * e).sum(-1)", "(du * v[t]).sum(-1)", ("dbeta",)),
    "dlog_a before the error's part": ("            dS = dS - kt[:, :, None] * dv[t][:, None, :]\n            dla[t] = (dS * old).sum((-1, -2))\n",
                                       "            dla[t] = (dS * old).sum((-1, -2))\n            dS = dS - kt[:, :, None] * dv[t][:, None, :]\n",
                                       ("dlog_a",)),
    "dlog_a of the next token": ("            dla[t] = (dS * old).sum((-1, -2))\n", "            dla[max(t - 1, lo)] = (dS * old).sum((-1, -2))\n", ("dlog_a",)),
    "gradient of the state not decayed": ("            dS = dS * np.exp(log_a[t])[:, None, None]\n", "", ("dk", "dv", "dinit")),
}


def as_outputs(want, dtype):
    return {n: torch.from_numpy(w).to(torch.float32 if n in FLOAT_OUTPUTS else DTYPE[dtype]) for n, w in want.items()}


def planted(name, d, scale):
    old, new, _ = MISTAKES[name]
    source = inspect.getsource(od)
    assert source.count(old) == 1, name
    copy = {}
    exec(compile(source.replace(old, new), "planted", "exec"), copy)
    args = [f64(d[n]) for n in ("q", "k", "v", "log_a", "beta")] + [d["cu"].numpy(), scale]
    y, final = copy["forward"](*args, f64(d["init"]))
    return dict(y=y, final=final, **copy["backward"](*args, f64(d["dy"]), f64(d["init"]), f64(d["dfinal"])))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("name", list(MISTAKES))
def test_a_planted_mistake_is_refused(name, dtype):
    d = make(4, [40, 0, 70], 4, 2, 32, 32, dtype)
    want = reference(d)
    check(as_outputs(want, dtype), want, d, dtype, "the model itself")
    wrong = planted(name, d, 32 ** -0.5)
    for n in MISTAKES[name][2]:
        with pytest.raises(AssertionError):
            check(as_outputs(dict(want, **{n: wrong[n]}), dtype), want, d, dtype, "%s in %s" % (name, n))
