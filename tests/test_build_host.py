"""The build's check of the registers that the pair kernels share out."""
import pytest

from fsdp_sharded_state_gb300 import build as fb

PAIR = "_ZN4fsdp86_GLOBAL__N__x8k_linearINS0_6LinCfgILi0EtLi2ELi256ELi1ELi0ELb0ELi4ELb0EEEEEv14CUtensorMap_stS4_NS0_8LinShapeENS_6LinEpiEm"
SPLIT = "_ZN4fsdp86_GLOBAL__N__x8k_linearINS0_6LinCfgILi0EtLi1ELi64ELi1ELi0ELb1ELin1ELb0EEEEEv14CUtensorMap_stS4_NS0_8LinShapeENS_6LinEpiEm"


def log(*kernels):
    return "".join(f"ptxas info    : Compiling entry function '{name}' for 'sm_103a'\nptxas info    : Function properties for {name}\n"
                   f"    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
                   f"ptxas info    : Used {n} registers, used 2 barriers\nptxas info    : Compile time = 9.0 ms\n" for name, n in kernels)


def test_pair_kernels_with_their_registers_pass():
    fb.check_pair_registers(log((PAIR, 168), (SPLIT, 96), ("_Z5otherv", 255)))
    fb.check_pair_registers("")


@pytest.mark.parametrize("n", [160, 170])
def test_another_count_fails_the_build(n):
    with pytest.raises(RuntimeError, match=f"k_linear.* {n} registers"):
        fb.check_pair_registers(log((SPLIT, 96), (PAIR, n), (PAIR, 168)))


def test_no_object_with_another_count_stays(tmp_path, monkeypatch):
    """A build that is refused leaves nothing that the next one would take for built."""
    class Result:
        returncode, stderr = 0, ""

        def __init__(self, out):
            self.stdout = out

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("object")
        return Result(log((PAIR, 160)) if "linear_" in out else "")

    monkeypatch.setattr(fb, "OUT", str(tmp_path))
    monkeypatch.setattr(fb, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(fb.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="160 registers"):
        fb.build()
    left = {p.name for p in tmp_path.iterdir()}
    assert "api.cu.o" in left and not any(n.startswith("linear_") for n in left) and "lib.so" not in left
