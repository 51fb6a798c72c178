"""The Muon step's driver on the CPU, its calls recorded in place of the library's:
what each stage is handed, and what two steps share."""
import torch

from zero_sharded_optimizer_reduce_amd import drivers


def _recorded(monkeypatch):
    calls = []
    for name in [n for n in vars(drivers) if n.startswith("zero_")]:
        if name in ("zero_shard_layout", "zero_newton_schulz_workspace"):
            continue
        monkeypatch.setattr(drivers, name, lambda *a, _name=name, **kw: calls.append((_name, a, kw)))
    return calls


def _storages(call):
    """Where the tensors of a call lie."""
    out = set()
    for a in list(call[1]) + list(call[2].values()):
        for t in a if isinstance(a, (list, tuple)) else [a]:
            if isinstance(t, torch.Tensor):
                out.add(t.untyped_storage().data_ptr())
    return out


def test_clipped_steps_share_no_memory(monkeypatch):
    # Two units' steps may run on two streams, or one be replayed from a graph
    # while the other runs: nothing that one writes may be the other's, and the
    # norm whose partial sums lie in one array per GPU may not be used.
    calls = _recorded(monkeypatch)
    steps = [drivers.MuonStep([(8, 24), (8, 24)], 2, device="cpu") for _ in range(2)]
    contributions = [[torch.zeros(st.psi_pad, dtype=torch.bfloat16) for _ in range(2)] for st in steps]
    used = []
    for st, grads in zip(steps, contributions):
        for _ in range(2):
            del calls[:]
            st.step(grads, [0.5, 0.5], dict(lr=1e-2, momentum=0.9), max_norm=1.0)
        names = [c[0] for c in calls]
        assert "zero_grad_norm_sq_no_alloc" not in names
        norm = calls[names.index("zero_grad_norm_sq")]
        shards, workspace, norm_sq, max_norm, clip = norm[1][:5]
        assert workspace.dtype == torch.float64 and workspace.numel() >= len(shards) * 1024
        assert norm_sq.dtype == torch.float64 and clip.dtype == torch.float32 and max_norm == 1.0
        moves = [c for c in calls if c[0] == "zero_muon_momentum"]
        assert len(moves) == 2 and all(c[2]["grad_scale"] is clip for c in moves)
        used.append(set().union(*map(_storages, calls)))
    assert not used[0] & used[1]


def test_a_clipped_step_allocates_only_once(monkeypatch):
    calls = _recorded(monkeypatch)
    st = drivers.MuonStep([(8, 24)], 1, device="cpu")
    grads = [torch.zeros(st.psi_pad, dtype=torch.bfloat16)]
    seen = []
    for _ in range(3):
        del calls[:]
        st.step(grads, [1.0], dict(lr=1e-2, momentum=0.9), max_norm=1.0)
        seen.append(set().union(*map(_storages, calls)))
    assert seen[0] == seen[1] == seen[2]
