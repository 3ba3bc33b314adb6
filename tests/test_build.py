"""The build asks for one compiler."""
import os

from mxfp8_mxfp4_experts_amd import build


def test_argument_checks_are_built_by_hipcc(monkeypatch, tmp_path):
    """The binding's argument checks need no compiler besides the library's."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return 0, ""
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "ARGS_OUT", str(tmp_path / "_tensor_args.so"))
    assert os.path.exists(build.build_args())
    assert [c[0] for c in ran] == [build.HIPCC]
