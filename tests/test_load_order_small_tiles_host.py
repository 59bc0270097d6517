"""The loads of the small tiles, whose waits count them (no GPU: the sources are
compiled to assembly).

A workgroup has up to three stages of loads to LDS on their way.  Before a barrier a
wave waits until at most one stage's are (two stages' before the first), and reads
behind it what the older ones brought.  So between two barriers that a stage's
products stand between there must be exactly one stage's loads to LDS, or none, and
no load to registers before them; a wave counts its loads in the order it starts
them, so that others behind them only make it wait longer."""
import re
import subprocess

import pytest

from param_collectives_amd import build

# (source, kernel): the instances of it
KERNELS = {("gated_block.hip", r"\d+gated_kernelILb[01]ELb1ELi64E"): 4, ("gated_block.hip", r"gated_grad_kernel.*Li64E"): 2,
           ("orthogonalize.hip", r"\d+symmetric_kernel.*Li64E"): 2, ("orthogonalize.hip", r"\d+update_kernel.*Li64E"): 2}


@pytest.fixture(scope="module")
def segments(tmp_path_factory):
    """{kernel: its instructions between barriers, in order: "L" a load to LDS, "r" one
    to registers, "m" a product, a number the loads that a wait leaves}, of a source."""
    kept = {}

    def of(source):
        if source in kept:
            return kept[source]
        path = tmp_path_factory.mktemp("asm") / "out.s"
        subprocess.run([build.hipcc(), *build.FLAGS, "--offload-device-only", "-S", f"{build.CSRC}/{source}", "-o",
                        str(path)], check=True)
        found, name = {}, None
        for line in path.read_text().splitlines():
            label = re.match(r"(_Z\w+):", line)
            if label:
                name = label.group(1)
                found[name] = [[]]
            elif line.startswith(".Lfunc_end"):
                name = None
            elif name and line.split():
                op = line.split()[0]
                if op == "s_barrier":
                    found[name].append([])
                elif re.match(r"(global|buffer|flat|scratch)_load", op):
                    found[name][-1].append("L" if re.search(r"\blds\b|_lds_", line) else "r")
                elif op.startswith("v_mfma"):
                    found[name][-1].append("m")
                elif op == "s_waitcnt" and "vmcnt" in line:
                    found[name][-1].append(int(re.search(r"vmcnt\((\d+)\)", line).group(1)))
        kept[source] = found
        return found

    return of


@pytest.mark.parametrize("source,kernel", KERNELS)
def test_a_stages_loads_between_barriers(segments, source, kernel):
    found = {n: s for n, s in segments(source).items() if re.search(kernel, n)}
    assert len(found) == KERNELS[source, kernel], list(found)
    for name, parts in found.items():
        # two stages' loads may be left before the first barrier, one stage's before the others
        first = [p for p in parts if "L" in p and "m" not in p and p[-1:] and isinstance(p[-1], int) and p[-1] > 0]
        assert first and first[0][-1] % 2 == 0, (name, parts)
        loads = first[0][-1] // 2
        loading = [p for p in parts if "m" in p and "L" in p]
        assert len(loading) >= 4, (name, parts)
        for p in loading:
            assert p.count("L") == loads, (name, p)
            last = len(p) - 1 - p[::-1].index("L")
            assert "r" not in p[:last], (name, p)
            # nothing is waited for among the products
            assert not any(isinstance(w, int) for w in p[:last]), (name, p)
            ends = [w for w in p[last:] if isinstance(w, int)]
            assert all(w in (0, loads) for w in ends), (name, p)
