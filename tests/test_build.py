"""What build() links anew."""
import os

from paged_kv_decode_v2_gb300 import build as b


def test_binding_of_another_torch_is_linked_anew(monkeypatch, tmp_path):
    """Built for one torch, then another, then the first again: its object is older than the link to the other."""
    for name, value in (("BUILD", tmp_path), ("LIB", tmp_path / "lib.so"), ("BIND", tmp_path / "bind.so")):
        monkeypatch.setattr(b, name, str(value))
    (tmp_path / "lib.so").touch()
    monkeypatch.setattr(b, "_sources", lambda: [])
    objects = {v: tmp_path / f"pa_bind-{v}.o" for v in ("1", "2")}
    for i, o in enumerate(objects.values()):
        o.touch()
        os.utime(o, (1000 + i, 1000 + i))
    linked = []

    def link(obj):
        linked.append(os.path.basename(obj))
        (tmp_path / "bind.so").touch()

    monkeypatch.setattr(b, "_link_bind", link)
    for version in ("1", "1", "2", "2", "1", "1"):
        monkeypatch.setattr(b, "_compile_bind", lambda force: str(objects[version]))
        b.build()
    assert linked == ["pa_bind-1.o", "pa_bind-2.o", "pa_bind-1.o"]
