"""The package's public names are the binding's, whatever the binding holds under them."""
import memory_bound_row_softmax_gb300 as pkg
from memory_bound_row_softmax_gb300 import binding


def test_a_replaced_function_is_reached_through_the_package(monkeypatch):
    first = pkg.status_string
    assert first is binding.status_string
    monkeypatch.setattr(binding, "status_string", lambda status: "replaced")
    assert pkg.status_string(0) == "replaced"
    monkeypatch.undo()
    assert pkg.status_string is first


def test_a_function_set_in_the_package_stays(monkeypatch):
    def mine(status):
        return "mine"
    pkg.status_string
    monkeypatch.setattr(pkg, "status_string", mine)
    monkeypatch.setattr(binding, "status_string", lambda status: "replaced")
    assert pkg.status_string is mine


def test_names():
    for name in pkg._BINDING_NAMES:
        assert getattr(pkg, name) is getattr(binding, name)
    try:
        pkg.no_such_name
    except AttributeError as e:
        assert "no_such_name" in str(e)
    else:
        raise AssertionError("an unknown name was found")
