"""The C library is built where torch is missing; only the Python binding, which
is compiled against it, is left out.  No compiler runs here."""
import os
import subprocess

from block_scaled_fp4_reduce_amd import build


class Done:
    def wait(self):
        return 0


def run(monkeypatch, tmp_path, torch):
    commands = []

    def made(cmd, *a, **k):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfp4q.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(subprocess, "Popen", made)
    monkeypatch.setattr(subprocess, "check_call", made)
    if not torch:
        find = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec",
                            lambda n, *a: None if n == "torch" else find(n, *a))
    assert build.build() == build.LIB
    return commands, sorted(os.listdir(tmp_path))


def test_without_torch(monkeypatch, tmp_path, capsys):
    commands, files = run(monkeypatch, tmp_path, torch=False)
    assert files == ["libfp4q.so"] and len(commands) == 3
    assert "torch" in capsys.readouterr().out


def test_with_torch(monkeypatch, tmp_path):
    commands, files = run(monkeypatch, tmp_path, torch=True)
    assert files == ["_calls.so", "libfp4q.so"] and len(commands) == 4
