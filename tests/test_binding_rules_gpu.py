"""The checks of _smla.so and those in Python say the same: whatever one takes the other takes,
argument by argument in unusual forms."""

import pytest
import torch

import sparse_mla_decode_csr_gb300 as smla
from test_paged_gpu import DEV, Batch
from test_paged_tree_gpu import step_state

pytestmark = pytest.mark.gpu


def forms(x):
    """Unusual forms of an argument, by name.  Their values are those of x or zeros: boundaries,
    lengths and pages that stay inside the tensors, as the kernels clamp them in any case."""
    if not torch.is_tensor(x):
        return {"none": None, "text": "x", "number": 0.25, "zero": 0, "huge": 1e300, "nan": float("nan"), "true": True}
    zeros = lambda *shape, dtype=x.dtype: torch.zeros(*shape, dtype=dtype, device=DEV)
    shape = list(x.shape)
    found = {"none": None, "number": 1.0, "host": x.cpu(), "double": zeros(*shape, dtype=torch.float64),
             "half": zeros(*shape, dtype=torch.float16), "int": zeros(*shape, dtype=torch.int32),
             "long": zeros(*shape, dtype=torch.int64), "byte": zeros(*shape, dtype=torch.uint8),
             "flat": x.reshape(-1), "deeper": x[None], "empty": zeros(*[0] * x.dim()), "sparse": zeros(*shape).to_sparse()}
    for d in range(x.dim()):
        for n in (0, shape[d] - 1, shape[d] + 1):
            if n >= 0 and not (n > shape[d] and x.dtype == torch.uint8):
                found[f"dim {d} of {n}"] = zeros(*shape[:d], n, *shape[d + 1:])
        found[f"dim {d} spread"] = zeros(*shape[:d], 2 * shape[d], *shape[d + 1:])[(slice(None),) * d + (slice(None, None, 2),)]
        found[f"dim {d} padded"] = zeros(*shape[:d], shape[d] + 8, *shape[d + 1:]).narrow(d, 0, shape[d])
        found[f"dim {d} off"] = zeros(*shape[:d], shape[d] + 1, *shape[d + 1:]).narrow(d, 1, shape[d])
        found[f"dim {d} repeated"] = zeros(*shape[:d], 1, *shape[d + 1:]).expand(*shape)
        if d:
            found[f"dim {d} first"] = zeros(*[shape[d]], *shape[:d], *shape[d + 1:]).movedim(0, d)
    return found


def calls(c, heads):
    """name -> (the call, its arguments in turn)."""
    s = step_state(c, heads, 6)
    ws = torch.zeros(smla.smla_paged_attend_workspace_size(max(c.rows, 1), heads, len(c.lens), 16, s["table"].shape[1]),
                     dtype=torch.uint8, device=DEV)
    batch = [s["kv"], s["table"], s["cu"], s["sl"]]
    q_out = s["q"][..., 512:]
    return {
        "write": (lambda kv, t, cu, sl, a, b, st: smla.smla_paged_write(a, b, kv, t, cu, sl, status=st),
                  batch + [s["lat"], s["rope"], s["status"]]),
        "read": (lambda kv, t, cu, sl, a, b, st: smla.smla_paged_read(kv, t, cu, sl, a, b, status=st),
                 batch + [s["lat"].clone(), s["rope"].clone(), s["status"]]),
        "append": (lambda kv, t, cu, sl, a, b, turns, q, o, pos, il, sc, st:
                   smla.smla_paged_append(a, b, kv, t, cu, sl, turns, q_rope=q, q_out=o, positions=pos, interleaved=il,
                                          rope_scale=sc, status=st),
                   batch + [s["lat"], s["rope"], s["turns"], s["q_rope"], q_out, s["pos"], True, 1.0, s["status"]]),
        "tree": (lambda p, cu, sl, m, pos, st: smla.smla_paged_tree(p, cu, sl, m, pos, status=st),
                 [s["parents"], s["cu"], s["sl"], s["mask"], s["pos"], s["status"]]),
        "attend": (lambda kv, t, cu, sl, q, sc, sink, o, z, ca, st, w:
                   smla.smla_paged_attend(q, kv, t, cu, sl, sc, sink, o, z, causal=ca, status=st, workspace_tensor=w),
                   batch + [s["q"], 1 / 24, torch.zeros(heads, device=DEV), s["out"], s["lse"], True, s["status"], ws]),
        "attend_tree": (lambda kv, t, cu, sl, q, m, sc, sink, o, z, ca, st, w:
                        smla.smla_paged_attend_tree(q, kv, t, cu, sl, m, sc, sink, o, z, causal=ca, status=st, workspace_tensor=w),
                        batch + [s["q"], s["mask"], 1 / 24, torch.zeros(heads, device=DEV), s["out"], s["lse"], False,
                                 s["status"], ws]),
        "accept": (lambda kv, t, cu, sl, p, new, n, st: smla.smla_paged_accept(kv, t, cu, sl, p, new, n_rows=n, status=st),
                   batch + [s["path"], s["new"], c.rows, s["status"]]),
    }


class Nothing:
    def __getattr__(self, name):
        return lambda *args: False


@pytest.mark.parametrize("lens,heads", [([(5, 40), (3, 9)], 4), ([(1, 1)], 1)])
@pytest.mark.parametrize("name", ["write", "read", "append", "tree", "attend", "attend_tree", "accept"])
def test_both_take_the_same_calls(name, lens, heads, monkeypatch):
    native, answers = smla._native, []

    class Asked:
        def __getattr__(self, call):
            def ask(*args):
                answers.append(getattr(native, call)(*args))
                return answers[-1]
            return ask

    call, args = calls(Batch(lens, 16), heads)[name]
    unlike, taken = [], 0
    for i in range(len(args)):
        for what, x in forms(args[i]).items():
            these = [*args[:i], x, *args[i + 1:]]
            answers.clear()
            monkeypatch.setattr(smla, "_native", Asked())
            try:
                call(*these)
            except Exception:  # (what the checks in Python say of it comes next)
                pass
            monkeypatch.setattr(smla, "_native", Nothing())
            try:
                call(*these)
                fine = True
            except Exception:
                fine = False
            taken += fine
            # (a number of another kind may be left to Python, which converts it)
            if (answers == [True]) > fine or (fine and answers != [True] and not isinstance(x, float)):
                unlike.append((i, what, list(answers), fine))
    torch.cuda.synchronize()
    assert unlike == [] and taken > len(args)
